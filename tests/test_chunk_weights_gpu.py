"""The softmax weights of requests of few rows take part in the product with the
values to 2^-16, in sums that nearly cancel: there a result's own rounding to bf16
hides nothing of a weight's."""
import numpy as np
import pytest
import torch

from mixture_value_projection_amd import binding
from test_chunk_attention_gpu import DEV, BF16, FP8, i32

U8, U24 = 2.0 ** -8, 2.0 ** -24


class Cancelling:
    """Requests of one new token, a query head a key head: the values are moved so
    that each row's weighted sum is near 0, as near as their type allows."""

    def __init__(self, seed, lens, H, D, bs, dtype):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.bs, self.H, self.D = list(lens), bs, H, D
        B, mb = len(self.lens), max(-(-n // bs) for n in self.lens)
        need = [-(-n // bs) for n in self.lens]
        perm = torch.randperm(sum(need), generator=g).numpy()
        self.table = np.full((B, mb), -1)
        at = np.cumsum([0] + need)
        for b in range(B):
            self.table[b, :need[b]] = perm[at[b]:at[b + 1]]
        self.scale = D ** -0.5
        self.q = torch.randn(B, H, D, generator=g).to(BF16)
        self.ks = self.vs = None
        if dtype == FP8:
            self.ks, self.vs = (torch.full((H,), 2.0 ** -5) for _ in range(2))

        def stored(x, s):
            return x.to(dtype) if s is None else (x / s[:, None]).clamp(-448, 448).to(dtype)
        self.k = stored(torch.randn(sum(need), bs, H, D, generator=g), self.ks)
        self.v = torch.zeros(sum(need), bs, H, D).to(dtype)
        self.rows = []
        for b in range(B):
            p = np.arange(self.lens[b])
            slots = (self.table[b][p // bs], p % bs)
            self.rows.append(slots)
            w = self.weights(b)[0]
            x = torch.randn(len(p), H, D, generator=g, dtype=torch.float64)
            for _ in range(3):
                x = x - torch.einsum("hn,nhd->hd", w, x)
                x = self.wide(stored(x.float(), self.vs), self.vs)
            raw = stored(x.float(), self.vs)
            if dtype == FP8:
                self.v.view(torch.uint8)[slots] = raw.view(torch.uint8)
            else:
                self.v[slots] = raw

    @staticmethod
    def wide(x, s):
        x = x.float().double()
        return x if s is None else x * s.double()[:, None]

    def at(self, pool, b, s):
        raw = pool.view(torch.uint8)[self.rows[b]].view(FP8) if pool.dtype == FP8 else pool[self.rows[b]]
        return self.wide(raw, s)

    def weights(self, b, part=None):
        """Softmax weights [H, n] of the request's row, and the logits' error."""
        q, k = self.q[b].double(), self.at(self.k, b, self.ks)
        z = torch.stack([k[:, h] @ q[h] for h in range(self.H)]) * self.scale
        d = (self.D + 4) * U24 * self.scale * torch.stack(
            [k[:, h].abs() @ q[h].abs() for h in range(self.H)]).amax(1)
        e = torch.exp(z - z.amax(1, keepdim=True))
        rounded = e if part is None else part(e)
        return rounded / e.sum(1, keepdim=True), d

    def want(self, part=None):
        """(out, tolerance): logits' errors as everywhere, weights to 2^-16, the
        exponential to 2^-18, fp32 sums, and the result rounded to bf16."""
        out, tol = (torch.zeros(len(self.lens), self.H, self.D, dtype=torch.float64) for _ in range(2))
        for b, n in enumerate(self.lens):
            w, d = self.weights(b, part)
            v = self.at(self.v, b, self.vs)
            for h in range(self.H):
                out[b, h] = w[h] @ v[:, h]
                spread = w[h] @ v[:, h].abs()
                tol[b, h] = (U8 * out[b, h].abs() + 2.0 ** -134
                             + (2.0 ** -16 + 2 * d[h] + 2.0 ** -18 + 2 * n * U24) * spread)
        return out, tol


CASES = [
    # lens, H, D, bs, dtype
    (list(range(1, 41)), 4, 64, 16, BF16), (list(range(2, 40)), 2, 128, 16, BF16),
    (list(range(3, 38)), 1, 256, 24, BF16), (list(range(1, 41)), 8, 128, 16, FP8),
    (list(range(2, 36)), 3, 64, 8, FP8), (list(range(2, 36)), 2, 256, 16, FP8),
    ([9, 700], 4, 128, 16, BF16), ([1500], 1, 64, 16, BF16), ([1500], 1, 128, 16, FP8),
]


@pytest.mark.parametrize("lens,H,D,bs,dtype", CASES[:6])
def test_one_rounding_to_bf16_is_not_within_the_tolerance(lens, H, D, bs, dtype):
    """The reference with weights rounded once leaves the tolerance, with weights
    in two bf16 parts it does not (CPU)."""
    c = Cancelling(1, lens, H, D, bs, dtype)
    want, tol = c.want()

    def once(e):
        return e.float().to(BF16).double()

    def twice(e):
        return once(e) + once(e - once(e))
    assert float(((c.want(once)[0] - want).abs() > tol - U8 * want.abs()).double().mean()) > 0.3
    assert bool(((c.want(once)[0].to(BF16).double() - want).abs() > tol).any())
    assert bool(((c.want(twice)[0].to(BF16).double() - want).abs() <= tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("G", [1, 3, 16])
@pytest.mark.parametrize("lens,H,D,bs,dtype", CASES)
def test_few_rows(lens, H, D, bs, dtype, G):
    """(The query heads of a key head are alike, so that all of them cancel.)"""
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    c = Cancelling(1, lens, H, D, bs, dtype)
    want, tol = c.want()
    B = len(lens)
    out = binding.attention_chunk_paged(
        c.q.repeat_interleave(G, 1).to(DEV), c.k.to(DEV), c.v.to(DEV), i32(c.table), i32(np.array(lens) - 1), i32(lens),
        i32(np.arange(B + 1)), c.scale, k_scale=None if c.ks is None else c.ks.to(DEV),
        v_scale=None if c.vs is None else c.vs.to(DEV)).cpu().double()
    worst = float(((out.reshape(B, H, G, D) - want[:, :, None]).abs() / tol[:, :, None]).max())
    print(f"{B} requests, {G * H} heads over {H} of {D}: worst {worst:.3f} of the tolerance", flush=True)
    assert worst <= 1
