"""The random paged sequences of ``test_gpu_tree_attention``, with a check in
which NaN fails and what a row does not see widens no bound.

Bounds, for a row's out = sum p v / z, z = sum p, over the tokens that it sees,
with mean magnitude A = sum p |v| / z:
  * a weight (with V's scale in it, in front of 8-bit codes) is rounded to fp16 there,
    else to the dtype: half a step, at most 2^-11 or eps / 2 of A;
  * fp16 has half a subnormal step of 2^-25 as its floor. Weights are held so that the
    largest is at least 2^6: each of N tokens is off by at most 2^-31 of the largest
    weight times its own largest |v|, or, with scales in the weights, of the largest
    product of weight and |v|;
  * a score is a sum of D products in fp32 and two multiplications: off by at most
    (D + 4) 2^-24 of B = max |scale| sum |q k|, and e^s by that relative (and
    2^-22 (B + 4) of exp2 and its argument); in numerator and denominator, so twice;
  * N additions in fp32: N 2^-24 of A, numerator and denominator, so twice;
  * the result is rounded: eps / 2 of it.
"""
import numpy as np
import torch

from oracle import serve_oracle as S
from test_gpu_tree_attention import Case

U32 = 2.0 ** -24


class Strict(Case):
    def values(self, b, t):
        """V of cached token t of sequence b: (codes or values [heads, dim], scales [heads] or None)."""
        page, off = divmod(int(self.slots[b][t]), self.page)
        return self.cache.v[page, :, off], None if self.cache.v_scale is None else self.cache.v_scale[page, :, off]

    def multiply_v(self, b, t, by):
        """Makes V of a cached token `by` (a power of two) times as large."""
        v, s = self.values(b, t)
        (v if s is None else s).mul_(by)

    def check(self, out, lse, rows=None, which=None, held=None, but=()):
        """`held`: only the first so many cached tokens of a sequence are anywhere. `but`: new
        tokens that are not looked at."""
        eps16 = torch.finfo(self.dtype).eps / 2
        quantised = self.fmt != "16"
        epsp = 2.0 ** -11 if quantised else eps16
        at = 0
        for b, (length, n) in enumerate(zip(self.lens, self.news)):
            got = out[at:at + n].double().cpu().numpy()
            glse = lse[at:at + n].double().cpu().numpy()
            q = self.q[at:at + n].double().cpu().numpy()
            at += n
            if n == 0 or (which is not None and b not in which):
                continue
            see = S.tree_visible(length, n, None if rows is None else rows[b])
            see[:, held:] &= held is None
            k, v = self.dense(b)
            for i in set(range(n)) - set(but):
                t = np.flatnonzero(see[i])
                for h in range(self.hq):
                    what = (b, i, h)
                    if len(t) == 0:
                        assert not got[i, h].any() and np.isneginf(glse[i, h]), what
                        continue
                    kk, vv = k[t, h // (self.hq // self.hk)], v[t, h // (self.hq // self.hk)]
                    s = kk @ q[i, h] * self.scale
                    p = np.exp(s - s.max())
                    z = p.sum()
                    want, A = p @ vv / z, p @ np.abs(vv) / z
                    B = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(self.scale)
                    most = np.abs(vv).max(-1)
                    floor = (p * most).max() if quantised else most.max() if self.dtype == torch.float16 else 0.0
                    score = (self.D + 4) * U32 * B + 2.0 ** -22 * (B + 4)
                    N = length + 64
                    tol = (epsp + 2 * score + 2 * N * U32) * A + eps16 * np.abs(want) + \
                        N * 2.0 ** -31 * floor / z + torch.finfo(self.dtype).tiny
                    off = np.abs(got[i, h] - want)
                    assert (off <= tol).all(), (what, float((off / tol).max()))
                    wlse = s.max() + np.log(z)
                    assert abs(glse[i, h] - wlse) <= score + N * U32 + 4 * U32 * abs(wlse), what
