"""rf_prefix_attention with more KV heads than a grid has places along its second side (65,535), within the bounds that
decoderef.attention derives, for many heads at a time."""
import pytest
import torch

import decoderef as R
import test_prefix_attention_gpu as P

pytestmark = pytest.mark.gpu


def _want(q, k, v, scale):
    """One sequence's rows in order behind `k` and `v`'s first ones: q [n][H][G][hd], k, v [keys][H][hd] in 64 bits."""
    n, keys = q.shape[0], k.shape[0]
    seen = torch.arange(keys, device="cuda") <= keys - n + torch.arange(n, device="cuda")[:, None]
    s = torch.einsum("nhgd,khd->nhgk", q, k) * scale
    s = s.masked_fill(~seen[:, None, None], -torch.inf)
    lse = torch.logsumexp(s, -1)
    w = (s - lse[..., None]).exp()
    out, mag = torch.einsum("nhgk,khd->nhgd", w, v), torch.einsum("nhgk,khd->nhgd", w, v.abs())
    size = torch.einsum("nhgd,khd->nhgk", q.abs(), k.abs()).amax(-1)
    eps = q.shape[-1] * 2.0 ** -22 * scale * size + 2.0 ** -20
    return out, lse, (R.U8 + 2 * eps + 2.0 ** -19)[..., None] * mag + R.U8 * out.abs() + 1e-30, eps + 2.0 ** -19 + 2.0 ** -21 * lse.abs()


@pytest.mark.parametrize("B,n,H,G,hd,prefix,lens", [
    (2, 2, 3, 2, 64, 130, [4, 0]),                       # (the formula above against few heads)
    (1, 1, 65535, 1, 64, 5, [3]),
    (1, 1, 65536, 1, 64, 5, [3]),
    (1, 1, 65537, 2, 128, 5, [0]),
    (2, 3, 70001, 1, 64, 130, [4, 0]),
    (1, 200, 65539, 1, 64, 9, [3]),                      # two row tiles
])
def test_prefix_attention_of_very_many_heads(B, n, H, G, hd, prefix, lens):
    q, kp, vp, k, v, kd, vd = P._data(B, n, H, G, hd, prefix, lens, 3)
    scale = hd ** -0.5
    out, lse, st = P._call(q, kp, vp, P._ints([prefix]), k, v, kd, vd, P._ints(lens), None, scale, H)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for b in range(B):
        for h in range(0, H, 4096):                    # (in 64 bits, some heads at a time)
            s, t = slice(h, min(h + 4096, H)), slice(h * G, min(h + 4096, H) * G)
            keys, values = (torch.cat([x[:prefix, s], y[b, :lens[b], s], z[b, :, s]]).double()
                            for x, y, z in ((kp, k, kd), (vp, v, vd)))
            mine = q[b, :, t].double().view(n, -1, G, hd)
            want, ln, b_out, b_lse = _want(mine, keys, values, scale)
            assert R.within(out[b, :, t].view(mine.shape), want, b_out) <= 1.0
            assert R.within(lse[b, :, t].view(ln.shape), ln, b_lse) <= 1.0
