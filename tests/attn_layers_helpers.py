"""64-bit references and device buffers for the attention-layer operators' tests.

Every reference is written from the formulas in include/gdna.h with numpy in 64
bits.  Caches are poisoned with NaN wherever no token lives, tables with page
numbers far outside the cache wherever no page is held, and outputs lie between
sentinel rows."""
import numpy as np
import torch

import gated_deltanet_linear_16_gb300 as gdn

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}   # relative, of normal values
HALF_STEP0 = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0, "e4m3": 2.0 ** -10}             # absolute, of subnormals
E32 = 2.0 ** -24
NOWHERE = 1 << 30


def f64(x):
    """A tensor's values in 64 bits on the host."""
    if x.dtype == torch.float8_e4m3fn:
        x = x.to(torch.float32)
    return x.double().cpu().numpy()


def raw_bytes(x):
    return x.contiguous().view(torch.uint8).cpu().numpy()


class Cache:
    """K and V arrays of a paged cache in one of several layouts, all NaN."""

    def __init__(self, pages, page, nkv, d, kind, layout="tokens", shift=0):
        self.pages, self.page, self.nkv, self.d, self.kind, self.layout = pages, page, nkv, d, kind, layout
        t = TYPES[kind]
        if layout == "tokens":                       # [pages, page, heads, d]
            shape, strides = (pages, page, nkv, d), (page * nkv * d, nkv * d, d)
            size = pages * page * nkv * d
            offset_v = size + 16
        elif layout == "heads":                      # [pages, heads, page, d]
            strides = (page * nkv * d, d, page * d)
            size = pages * page * nkv * d
            offset_v = size + 16
        elif layout == "pair":                       # [pages, 2, page, heads, d]
            strides = (2 * page * nkv * d, nkv * d, d)
            size = 2 * pages * page * nkv * d
            offset_v = page * nkv * d
        elif layout == "beside":                     # [pages, page, heads, 2, d]
            strides = (2 * page * nkv * d, 2 * nkv * d, 2 * d)
            size = 2 * pages * page * nkv * d
            offset_v = d
        else:                                        # "padded": room after each head, token and page
            strides = ((page * (nkv * (d + 16) + 16) + 32), nkv * (d + 16) + 16, d + 16)
            size = pages * strides[0]
            offset_v = size + 16
        self.page_stride, self.token_stride, self.head_stride = strides
        self.shift = shift
        total = offset_v + size + 64 + shift
        if kind == "e4m3":
            self.buf = torch.full((total,), 0x7F, dtype=torch.uint8, device="cuda").view(t)
        else:
            self.buf = torch.full((total,), float("nan"), dtype=t, device="cuda")
        self.k = self.buf[shift:].as_strided((pages, page, nkv, d), strides + (1,))
        self.v = self.buf[shift + offset_v:].as_strided((pages, page, nkv, d), strides + (1,))

    def addresses(self):
        return self.k.data_ptr(), self.v.data_ptr()

    def args(self):
        return dict(pages=self.pages, page_size=self.page, page_stride=self.page_stride,
                    token_stride=self.token_stride, head_stride=self.head_stride,
                    cache_dtype={"f16": gdn.GDNA_F16, "bf16": gdn.GDNA_BF16, "e4m3": gdn.GDNA_E4M3}[self.kind])

    def put(self, which, page, token, x):
        """x [n, nkv, d] float32 (CPU) at (page[i], token[i]), rounded to the cache's type; returns the stored values."""
        t = x.to(TYPES[self.kind])
        dst = getattr(self, which)
        at = (torch.as_tensor(page, device="cuda"), torch.as_tensor(token, device="cuda"))
        if self.kind == "e4m3":
            dst.view(torch.uint8)[at] = t.view(torch.uint8).cuda()
        else:
            dst[at] = t.cuda()
        return f64(t)


def guarded(rows, length, stride, kind, before=5):
    """A [rows, stride] output between sentinel elements; returns (whole, view of the rows' payload)."""
    t = TYPES[kind]
    whole = torch.full((before + rows * stride + 7,), 77.0, dtype=t, device="cuda")
    return whole, whole[before:before + rows * stride].view(rows, stride)[:, :length]


def intact(whole, view):
    """Everything of `whole` outside `view` still holds the sentinel."""
    probe = whole.clone()
    start = (view.data_ptr() - whole.data_ptr()) // whole.element_size()
    probe[start:].as_strided(view.shape, view.stride()).fill_(77.0)
    return bool((probe == 77.0).all())


def rotate64(x, cos, sin, rot, interleaved):
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        h = rot // 2
        a, b = x[..., :h], x[..., h:rot]
        y[..., :h], y[..., h:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def attention64(q, keys, values, lens, q_len, scale, gate=None):
    """q [B*q_len, nq, d]; keys/values: per sequence [len, nkv, d].  Returns out, lse, and the sizes that the
    error bound needs: max_j sum_i |q_i k_ji| * scale and max |v| of each row."""
    rows, nq, d = q.shape
    out, lse = np.zeros((rows, nq, d)), np.full((rows, nq), -np.inf)
    size, vmax = np.zeros((rows, nq, 1)), np.zeros((rows, nq, 1))
    for r in range(rows):
        b, t = divmod(r, q_len)
        n = lens[b] - (q_len - 1 - t)
        if n <= 0:
            continue
        k, v = keys[b][:n], values[b][:n]
        g = nq // k.shape[1]
        for h in range(nq):
            s = (k[:, h // g] @ q[r, h]) * scale
            m = s.max()
            p = np.exp(s - m)
            out[r, h] = p @ v[:, h // g] / p.sum()
            lse[r, h] = m + np.log(p.sum())
            size[r, h] = (np.abs(k[:, h // g]) @ np.abs(q[r, h])).max() * scale
            vmax[r, h] = np.abs(v[:, h // g]).max()
    if gate is not None:
        out = out / (1 + np.exp(-gate))
    return out, lse, size, vmax
