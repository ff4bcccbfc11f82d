"""Random sequences of the paged cache's calls against the oracle: prompts, chunks with and without appending, branches,
truncations, single tokens, reading back, in caches that run out of pages, blocks and slots."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from bit_kivi_kv_gb300.kivi import KiviError, kivi_paged_set_max_ctas  # noqa: E402
from chunk_harness import ChunkRun, head_strided, in_wider, oracle_chunk  # noqa: E402


class Calls:
    def __init__(self, seed):
        self.rng = rng = random.Random(seed)
        self.D = rng.choice([64, 128])
        self.G = rng.choice([g for g in (32, 64, 128) if g <= self.D])
        self.R = self.G * rng.choice([1, 1, 2, 3])
        nq, Hkv = rng.choice([1, 2, 4]), rng.choice([1, 2, 3, 5])
        self.Hq, self.slots, self.pool = nq * Hkv, rng.randint(2, 9), rng.choice([6, 20, 60, 200])
        self.run = ChunkRun(self.Hq, Hkv, self.D, rng.choice([2, 4, 8]), self.G, self.R, max_seqs=self.slots,
                            max_blocks=rng.choice([4, 16, 64]), n_pages=self.pool, seed=seed, sink=rng.random() < 0.7)
        self.c = self.run.cache

    def room(self, call):
        """The call, or a refusal that changes nothing."""
        before = self.c.free(), [self.c.counts(s) for s in self.run.live]
        try:
            call()
        except KiviError:
            assert before == (self.c.free(), [self.c.counts(s) for s in self.run.live])

    def chunk(self):
        rng = self.rng
        seqs = rng.sample(list(self.run.live), rng.randint(1, len(self.run.live)))
        lens = [rng.choice([0, 1, 1, 2, 3, 4, 8, 16, 17, rng.randint(0, 70), rng.randint(0, 300)]) for _ in seqs]
        kw = {}
        if rng.random() < 0.3:
            kw["window"] = rng.choice([1, 5, 64, 200, 5000])
        if rng.random() < 0.2:
            kw["cap"] = rng.choice([1.0, 20.0, 50.0])
        if rng.random() < 0.2:
            kw["slopes"] = torch.tensor([rng.uniform(-0.01, 0.5) for _ in range(self.Hq)], device="cuda")
        return seqs, lens, self.run.chunk(lens), rng.choice([lambda x: x, head_strided, in_wider]), kw

    def told(self, seqs, lens, k, v):
        first = 0
        for s, n in zip(seqs, lens):
            part = slice(first, first + n)
            oracle_chunk(self.run.live[s], k[part].transpose(0, 1).cpu().numpy(), v[part].transpose(0, 1).cpu().numpy())
            first += n

    # -- the calls ------------------------------------------------------------------
    def add(self):
        G, R = self.G, self.R
        L = self.rng.choice([0, 1, G - 1, G, R, R + 1, self.rng.randint(0, 600), self.rng.randint(0, 3000)])
        self.room(lambda: self.run.add(L))

    def attend(self):
        seqs, lens, data, fit, kw = self.chunk()
        kivi_paged_set_max_ctas(self.c.handle, self.rng.choice([0, 0, 0, 1, 2, 5, 40]))
        self.run.attend(seqs, lens, data, fit=fit, **kw)
        kivi_paged_set_max_ctas(self.c.handle, 0)

    def append(self):
        seqs, lens, data, fit, _ = self.chunk()
        self.room(lambda: self.run.append(seqs, lens, data, fit=fit))

    def extend(self):
        seqs, lens, (q, k, v), fit, kw = self.chunk()

        def call():
            out = self.c.extend(seqs, lens, fit(q), fit(k), fit(v), **kw)
            self.run.check_out(seqs, lens, q, k, v, out, 0.0, kw.get("cap", 0.0), kw.get("window", 0), kw.get("slopes"))
            self.told(seqs, lens, k, v)
        self.room(call)

    def fork(self):
        seqs = [self.rng.choice(list(self.run.live)) for _ in range(self.rng.randint(1, 3))]

        def call():
            new = self.run.fork(seqs)
            for s, t in zip(seqs, new):
                if sum(self.c.counts(s)):
                    q = (1.5 * torch.randn(1, self.Hq, self.D, device="cuda")).half()
                    assert torch.equal(self.c.append_decode([t], None, None, q), self.c.append_decode([s], None, None, q))
        self.room(call)

    def truncate(self):
        s = self.rng.choice(list(self.run.live))
        quantized, rows = self.c.counts(s)
        self.run.truncate(s, self.rng.choice([quantized + self.rng.randint(0, rows),
                                              self.G * self.rng.randint(0, quantized // self.G)]))

    def release(self):
        self.run.release(self.rng.choice(list(self.run.live)))

    def single(self):
        seqs = self.rng.sample(list(self.run.live), self.rng.randint(1, len(self.run.live)))
        for _ in range(self.rng.choice([1, 2, 5])):
            q, k, v = self.run.chunk([1] * len(seqs))

            def call():
                if self.rng.random() < 0.5:
                    self.c.append(seqs, k, v)
                else:
                    self.c.append_decode(seqs, k, v, q)
                for i, s in enumerate(seqs):
                    self.run.live[s].append(k[i].cpu().numpy()[None], v[i].cpu().numpy()[None])
            self.room(call)

    def read(self):
        s = self.rng.choice(list(self.run.live))
        n = sum(self.c.counts(s))
        first = self.rng.randint(0, n)
        count = self.rng.randint(0, n - first)
        got = self.c.read([s], first, count)
        for x, hat in zip(got, (self.run.live[s].keys_hat(), self.run.live[s].values_hat())):
            assert torch.equal(x[0], torch.from_numpy(hat[0][:, first:first + count]).half().cuda())


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    t = Calls(seed)
    for step in range(40):
        name = t.rng.choice(["add", "add", "attend", "attend", "append", "append", "extend", "fork", "truncate", "release",
                             "single", "read"])
        if name == "add" or t.run.live:
            getattr(t, name)()
        if step % 4 == 0:
            t.run.check()
    t.run.check()
    for s in list(t.run.live):
        t.run.release(s)
    assert t.c.free() == (t.pool, t.slots)
