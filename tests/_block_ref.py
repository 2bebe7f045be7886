"""Plain 64-bit forms of the decoder-block operators (numpy), written from their formulas."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def quantise(v):
    """(codes 0..15, scale codes) of v [..., n] in MXFP4: nearest E2M1 value, ties to the even code."""
    v = np.asarray(v, dtype=np.float64)
    blocks = v.reshape(*v.shape[:-1], -1, 32)
    top = np.abs(blocks).max(-1)
    bad = ~np.isfinite(blocks).all(-1)
    safe = np.where(bad | (top == 0), 1.0, top)
    e = np.clip(np.floor(np.log2(safe)).astype(int), -200, 200)
    e += (np.exp2(e + 1.0) <= safe).astype(int) - (np.exp2(e.astype(float)) > safe).astype(int)
    e = np.where(top == 0, -127, np.clip(e - 2, -127, 127))
    a = np.abs(np.where(bad[..., None], 0.0, blocks)) / np.exp2(e.astype(float))[..., None]
    dist = np.abs(a[..., None] - E2M1)
    near = dist.min(-1, keepdims=True)
    codes = np.arange(8)
    # among equally near codes the even one
    pick = np.where(dist == near, codes + 100 * (codes % 2), 1000).argmin(-1)
    codes = (pick + 8 * np.signbit(blocks) * ~bad[..., None]).astype(np.uint8)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return codes.reshape(v.shape), scales


def values(codes, scales):
    c = codes.reshape(*codes.shape[:-1], -1, 32)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (np.where(c & 8, -1.0, 1.0) * E2M1[c & 7] * s[..., None]).reshape(codes.shape)


def rounded(v):
    return values(*quantise(v))


def row_major_bytes(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def pack_rows(codes, scales):
    """wd_fp4's packed arrays from codes [N, K] and scales [N, K / 32], element by element."""
    N, K = codes.shape
    rt, ct = -(-N // 16), -(-K // 128)
    pc = np.zeros((rt, ct, 16, 4, 4, 4), np.uint8)
    ps = np.zeros((rt, ct, 8, 2, 4), np.uint8)
    n, k = np.meshgrid(np.arange(N), np.arange(K), indexing="ij")
    at = (n // 16, k // 128, n % 16, k % 32 // 8, k % 128 // 32, k % 8 // 2)
    np.add.at(pc, at, codes << (4 * (k % 2)).astype(np.uint8))
    n, b = np.meshgrid(np.arange(N), np.arange(K // 32), indexing="ij")
    ps[n // 16, b // 4, n % 8, n % 16 // 8, b % 4] = scales
    return pc.reshape(-1), ps.reshape(-1)


def attend(q, k, v, scale):
    """out, lse, sum p|v| and the largest sum |q k| scale of q [heads, D] over k, v [keys, kv_heads, D]."""
    H, D = q.shape
    G = H // k.shape[1]
    out, lse, mag, reach = np.zeros((H, D)), np.full(H, -np.inf), np.zeros((H, D)), np.zeros(H)
    for h in range(H if k.shape[0] else 0):
        kk, vv = k[:, h // G], v[:, h // G]
        z = kk @ q[h] * scale
        top = z.max()
        p = np.exp(z - top)
        lse[h] = top + np.log(p.sum())
        p /= p.sum()
        out[h], mag[h] = p @ vv, p @ np.abs(vv)
        reach[h] = (np.abs(kk) @ np.abs(q[h])).max() * abs(scale)
    return out, lse, mag, reach


def norm(res, y, w_post, gate, w_pre, res_scale, eps):
    """r', out, and |res_scale res| + |gate n| (what r' is the difference of)."""
    def n(v, w):
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * w
    a = res_scale * res
    b = 0.0 * a if y is None else (n(y, w_post) if w_post is not None else y) * (1.0 if gate is None else gate)
    r = a + b
    return r, None if w_pre is None else n(r, w_pre), np.abs(a) + np.abs(b)
