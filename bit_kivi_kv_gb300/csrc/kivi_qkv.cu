// Norm of every query and key head, the position rotation and the change to
// the cache's layout in one pass over a projection's output (include/kivi.h,
// kivi_qk_norm_rope).
//
// Per head row x of D channels (q and k; v is only copied and rounded):
//   y = x / sqrt(mean(x^2) + eps) * w            with a weight, else y = x
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)   for the rotated pairs
//   out = fp16(y)
// All in fp32, rounded once.
//
// D / 8 lanes hold a row, each two runs of four channels that are each
// other's rotation partners (half-split pairs: c and c + rot / 2) or hold whole
// pairs (interleaved: 2j and 2j + 1), so the rotation needs no exchange and
// the norm one sum over D / 8 lanes.  A warp stays on one token and walks over
// heads of one tensor, with the token's cosines and sines and the weight in
// registers; the CTA's warps take consecutive tokens of the same heads, so
// that both the token-major reads and the head-major writes are runs of
// several rows.
#include <cuda_bf16.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <type_traits>

#include "kivi_blocks.cuh"
#include "kivi_decode_mma.cuh"

namespace kivi {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

kivi_status failf(kivi_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
kivi_status failf(kivi_status st, const char* fmt, ...) {
    char msg[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return report_error(st, msg);
}

constexpr int kWarps = 4;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kAhead = 2;     // groups of heads computed together, with the next ones' loads in flight

struct Part {                 // one of q, k, v
    const void* src;
    long long s_batch, s_token, s_head;   // elements
    __half* dst;
    long long d_slot;         // elements between (batch row, head) slots
    const float* w;           // null: no norm
    int heads;
    int chunks, passes;       // grid.y entries of this tensor, and the groups of heads each takes
    int turn;                 // rotated
};
struct Args {
    Part part[3];
    long long tokens, total;  // per batch row, in all
    const float* cos_sin;
    const void* positions;
    long long first_position, n_positions;
    int rot, wide;            // rotated channels; positions are 64-bit
    float eps;
};

// four channels as loaded, and as fp32
template <typename T>
struct Raw { using type = uint2; };
template <>
struct Raw<float> { using type = uint4; };
__device__ __forceinline__ void widen(const uint4& v, float (&x)[4], float) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void widen(const uint2& v, float (&x)[4], __half) {
    const float2 a = mma_detail::unpack_f16x2(v.x), b = mma_detail::unpack_f16x2(v.y);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
__device__ __forceinline__ void widen(const uint2& v, float (&x)[4], __nv_bfloat16) {   // bf16: fp32's upper half
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ uint2 ldg_raw(const void* p, uint2) { return mma_detail::ldg_stream2(p); }
__device__ __forceinline__ uint4 ldg_raw(const void* p, uint4) { return mma_detail::ldg_stream(p); }
__device__ __forceinline__ void store4(__half* p, const float (&x)[4]) {
    uint2 v;
    v.x = mma_detail::pack_f16x2(x[0], x[1]);
    v.y = mma_detail::pack_f16x2(x[2], x[3]);
    *reinterpret_cast<uint2*>(p) = v;
}

template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_kernel(const __grid_constant__ Args a) {
    constexpr int LPR = D / 8;            // lanes per row
    constexpr int RPW = 32 / LPR;         // rows a warp holds
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lr = lane % LPR, sub = lane / LPR;
    int chunk = blockIdx.y, which = 0;
    while (chunk >= a.part[which].chunks) chunk -= a.part[which++].chunks;
    const Part& p = a.part[which];
    const long long tok = (long long)blockIdx.x * kWarps + warp;
    mma_detail::griddepcontrol_wait();
    mma_detail::griddepcontrol_launch_dependents();
    if (tok >= a.total) return;
    const long long b = tok / a.tokens, t = tok % a.tokens;

    // the lane's two runs of four channels
    int ca, cb;
    const int rot = p.turn ? a.rot : 0;
    if (INTERLEAVED) {
        ca = 8 * lr;
        cb = ca + 4;
    } else if (8 * lr < rot) {
        ca = 4 * lr;
        cb = ca + rot / 2;
    } else {
        ca = rot + 4 * (lr - rot / 8);
        cb = ca + (D - rot) / 2;
    }
    const bool turned = 8 * lr < rot;
    const T* src = reinterpret_cast<const T*>(p.src) + b * p.s_batch + t * p.s_token;
    __half* dst = p.dst + b * p.heads * p.d_slot + t * D;
    const int h0 = chunk * p.passes * RPW + sub;
    // kAhead groups at a time, the next ones' loads before the present ones'
    // work; the first ones' go out ahead of the token's position and table row
    using V = typename Raw<T>::type;
    V xa[kAhead], xb[kAhead];
    auto fetch = [&](int it, V (&ya)[kAhead], V (&yb)[kAhead]) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = h0 + (it + u) * RPW;
            ya[u] = yb[u] = V{};
            if (it + u < p.passes && h < p.heads) {
                ya[u] = ldg_raw(src + h * p.s_head + ca, V{});
                yb[u] = ldg_raw(src + h * p.s_head + cb, V{});
            }
        }
    };
    fetch(0, xa, xb);
    float cs[4], sn[4];                   // interleaved: the four pairs of the eight channels
    if (turned) {
        long long pos = a.first_position + t;
        if (a.positions)
            pos = a.wide ? reinterpret_cast<const long long*>(a.positions)[tok]
                         : reinterpret_cast<const int*>(a.positions)[tok];
        if (pos >= 0 && pos < a.n_positions) {
            const float* tab = a.cos_sin + pos * rot + 4 * lr;
            const float4 c = *reinterpret_cast<const float4*>(tab);
            const float4 s = *reinterpret_cast<const float4*>(tab + rot / 2);
            cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
            sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
        } else {                          // a position without a table row: the token's heads become NaN
#pragma unroll
            for (int j = 0; j < 4; ++j) cs[j] = sn[j] = NAN;
        }
    }
    float wa[4], wb[4];
    if (p.w) {
        widen(*reinterpret_cast<const uint4*>(p.w + ca), wa, 0.f);
        widen(*reinterpret_cast<const uint4*>(p.w + cb), wb, 0.f);
    }
    for (int it = 0; it < p.passes; it += kAhead) {
        V na[kAhead], nb[kAhead];
        fetch(it + kAhead, na, nb);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = h0 + (it + u) * RPW;
            float ya[4], yb[4];
            widen(xa[u], ya, T{});
            widen(xb[u], yb, T{});
            if (p.w) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) s = fmaf(ya[j], ya[j], fmaf(yb[j], yb[j], s));
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
                const float ms = s * (1.0f / D) + a.eps;
                float r = 1.0f / sqrtf(ms);
                // squares that leave fp32's range (values above 2^63, or below 2^-50
                // with next to no eps; not fp16's): the row times a power of two of its
                // largest value.  One unsigned comparison: not in [2^-100, 2^126).
                const bool far = !std::is_same<T, __half>::value && __float_as_uint(ms) - 0x0d800000u >= 0x71000000u;
                if (__any_sync(kFull, far)) {
                    float most = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) most = fmaxf(most, fmaxf(fabsf(ya[j]), fabsf(yb[j])));
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
                    const int e = max(-126, min(126, (int)(__float_as_uint(most) >> 23) - 127));
                    const float c = far ? mma_detail::pow2i(-e) : 1.f;
                    s = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        ya[j] *= c;
                        yb[j] *= c;
                        s = fmaf(ya[j], ya[j], fmaf(yb[j], yb[j], s));
                    }
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
                    if (far) r = 1.0f / sqrtf(s * (1.0f / D) + a.eps * c * c);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ya[j] = ya[j] * r * wa[j];
                    yb[j] = yb[j] * r * wb[j];
                }
            }
            if (turned) {
                if (INTERLEAVED) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float x0 = ya[2 * j], x1 = ya[2 * j + 1];
                        ya[2 * j] = x0 * cs[j] - x1 * sn[j];
                        ya[2 * j + 1] = x1 * cs[j] + x0 * sn[j];
                        const float x2 = yb[2 * j], x3 = yb[2 * j + 1];
                        yb[2 * j] = x2 * cs[2 + j] - x3 * sn[2 + j];
                        yb[2 * j + 1] = x3 * cs[2 + j] + x2 * sn[2 + j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x0 = ya[j], x1 = yb[j];
                        ya[j] = x0 * cs[j] - x1 * sn[j];
                        yb[j] = x1 * cs[j] + x0 * sn[j];
                    }
                }
            }
            if (it + u < p.passes && h < p.heads) {
                __half* row = dst + h * p.d_slot;
                store4(row + ca, ya);
                store4(row + cb, yb);
            }
            xa[u] = na[u];
            xb[u] = nb[u];
        }
    }
}

template <typename T, int D>
cudaError_t launch_t(Args& a, int interleaved, cudaStream_t st) {
    constexpr int RPW = 256 / D;
    // Groups of heads a warp walks over: as many as leave about 8192 warps (one
    // wave of the GPU), 2 to 16, the same number in all chunks of a tensor.  A
    // long walk spreads the token's table row and keeps loads in flight (7B prompt,
    // 96 heads x 32768 tokens: 2 groups 371 us, 16 groups 252 us); a short one
    // fills the GPU (2331 tokens of 32 heads: 2 groups 7.1 us, 16 groups 15.6 us).
    long long groups = 0;
    for (const Part& p : a.part) groups += (p.heads + RPW - 1) / RPW;
    const long long fit = groups * a.total / 8192;
    const int most = fit < 2 ? 2 : fit > 16 ? 16 : (int)fit;
    int chunks = 0;
    for (Part& p : a.part) {
        const int n = (p.heads + RPW - 1) / RPW;
        p.chunks = (n + most - 1) / most;
        p.passes = p.chunks ? (n + p.chunks - 1) / p.chunks : 0;
        chunks += p.chunks;
    }
    const long long ctas = (a.total + kWarps - 1) / kWarps;
    if (ctas > 0x7fffffffLL || chunks > 65535) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)ctas, (unsigned)chunks);
    return interleaved ? launch_dependent(qk_norm_rope_kernel<T, D, true>, grid, 32 * kWarps, st, a)
                       : launch_dependent(qk_norm_rope_kernel<T, D, false>, grid, 32 * kWarps, st, a);
}

}  // namespace

kivi_status check_qkv(const kivi_qkv* a) {
    if (!a) return failf(KIVI_ERR_INVALID_ARG, "null arguments");
    if (a->batch < 0 || a->n_tokens < 0) return failf(KIVI_ERR_INVALID_ARG, "negative batch or token count");
    if (a->n_q_heads < 1 || a->n_kv_heads < 1) return failf(KIVI_ERR_INVALID_ARG, "head counts must be positive");
    if (a->head_dim != 64 && a->head_dim != 128) return failf(KIVI_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (a->n_q_heads > 8192 || a->n_kv_heads > 8192) return failf(KIVI_ERR_UNSUPPORTED, "head counts must be <= 8192");
    if (a->batch > 0 && a->n_tokens > (1LL << 32) / a->batch)
        return failf(KIVI_ERR_UNSUPPORTED, "batch * n_tokens must be <= 2^32");
    if (a->dtype != KIVI_F16 && a->dtype != KIVI_BF16 && a->dtype != KIVI_F32)
        return failf(KIVI_ERR_INVALID_ARG, "unknown input type %d", a->dtype);
    if (a->batch > 0 && a->n_tokens > 0 && !a->q && !a->k && !a->v)   // (empty tensors have null addresses)
        return failf(KIVI_ERR_INVALID_ARG, "q, k and v are all null");
    const int size = a->dtype == KIVI_F32 ? 4 : 2;
    const struct { const char* name; const void* src; const long long* stride; } in[3] = {
        {"q", a->q, a->q_stride}, {"k", a->k, a->k_stride}, {"v", a->v, a->v_stride}};
    for (const auto& t : in) {
        if (!t.src) continue;
        if (!aligned(t.src, 16)) return failf(KIVI_ERR_INVALID_ARG, "%s must be 16-byte aligned", t.name);
        for (int j = 0; j < 3; ++j)
            if (t.stride[j] * size % 16)
                return failf(KIVI_ERR_INVALID_ARG, "%s's strides must be multiples of 16 bytes", t.name);
    }
    if (!(a->eps >= 0.f) || isinf(a->eps)) return failf(KIVI_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!aligned(a->q_weight, 16) || !aligned(a->k_weight, 16))
        return failf(KIVI_ERR_INVALID_ARG, "the weights must be 16-byte aligned");
    if (a->cos_sin) {
        if (a->rot_dim < 8 || a->rot_dim > a->head_dim || a->rot_dim % 8)
            return failf(KIVI_ERR_INVALID_ARG, "rot_dim must be a multiple of 8 in [8, head_dim]");
        if (a->n_positions < 1) return failf(KIVI_ERR_INVALID_ARG, "n_positions must be positive");
        if (!aligned(a->cos_sin, 16)) return failf(KIVI_ERR_INVALID_ARG, "cos_sin must be 16-byte aligned");
        if (!aligned(a->positions, a->positions_64bit ? 8 : 4))
            return failf(KIVI_ERR_INVALID_ARG, "positions must be aligned to their size");
    }
    return KIVI_OK;
}

cudaError_t launch_qk_norm_rope(const kivi_qkv& q, const QkvDest& d, cudaStream_t st) {
    Args a{};
    const bool turn = q.cos_sin != nullptr;
    auto part = [](const void* src, const long long* s, __half* dst, long long slot, const float* w, int heads, int t) {
        return Part{src, s[0], s[1], s[2], dst, slot, w, src ? heads : 0, 0, 0, t};
    };
    a.part[0] = part(q.q, q.q_stride, d.q, d.q_slot, q.q_weight, q.n_q_heads, turn);
    a.part[1] = part(q.k, q.k_stride, d.k, d.k_slot, q.k_weight, q.n_kv_heads, turn);
    a.part[2] = part(q.v, q.v_stride, d.v, d.v_slot, nullptr, q.n_kv_heads, 0);
    a.tokens = q.n_tokens;
    a.total = q.batch * q.n_tokens;
    a.cos_sin = q.cos_sin;
    a.positions = q.positions;
    a.first_position = q.first_position;
    a.n_positions = q.n_positions;
    a.rot = turn ? q.rot_dim : 0;
    a.wide = q.positions_64bit;
    a.eps = q.eps;
#define KIVI_N(CODE, T)                                                                                  \
    if (q.dtype == CODE)                                                                                 \
        return q.head_dim == 128 ? launch_t<T, 128>(a, q.interleaved, st) : launch_t<T, 64>(a, q.interleaved, st);
    KIVI_N(KIVI_F16, __half) KIVI_N(KIVI_BF16, __nv_bfloat16) KIVI_N(KIVI_F32, float)
#undef KIVI_N
    return cudaErrorInvalidValue;
}

}  // namespace kivi

extern "C" kivi_status kivi_qk_norm_rope(const kivi_qkv* a, kivi_stream_t stream) {
    using namespace kivi;
    const kivi_status st = check_qkv(a);
    if (st != KIVI_OK) return st;
    if ((a->q && !a->q_out) || (a->k && !a->k_out) || (a->v && !a->v_out))
        return failf(KIVI_ERR_INVALID_ARG, "an input without its output");
    if (!aligned(a->q_out, 16) || !aligned(a->k_out, 16) || !aligned(a->v_out, 16))
        return failf(KIVI_ERR_INVALID_ARG, "the outputs must be 16-byte aligned");
    if (a->batch == 0 || a->n_tokens == 0) return report_error(KIVI_OK, "");
    const long long slot = a->n_tokens * a->head_dim;
    const QkvDest d{static_cast<__half*>(a->q_out), static_cast<__half*>(a->k_out), static_cast<__half*>(a->v_out),
                    slot, slot, slot};
    const cudaError_t e = launch_qk_norm_rope(*a, d, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return failf(KIVI_ERR_CUDA, "norm and rotation launch: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    count_launches(1);
    return report_error(KIVI_OK, "");
}
