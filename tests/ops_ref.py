"""Plain 64-bit references of the few-token layer and the dense product, with the
elementwise error that fp32 arithmetic may leave.

Every bound below is worst-case arithmetic, not a measurement.  A sum of n products in
fp32, in any order and grouping, is off by at most (n + 2) 2^-24 times the sum of the
products' magnitudes (each product and each addition rounds by 2^-24 relative, or is exact
in a fused step).  A chain of such steps adds up their bounds; `STEPS` more roundings cover
the scales, the bias, the residual and the exponential of the activation (a few units in
the last place).  The final rounding adds half a step of y's format, relative to y."""
import math

import numpy as np
import torch

import synth

U = 2.0 ** -24
TINY = 2.0 ** -126  # below the smallest normal number a product or a result loses its bits altogether
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
STEPS = 16


def act(v, name):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


ACT_SLOPE = 1.13  # largest |derivative| of SiLU (1.0998) and of tanh-GELU (1.129); 1 without one


def weights(rows, cols, wfmt, seed, std=0.05):
    """Stored weights and their values: (W, s, float64 [rows, cols]) as torch CPU tensors."""
    if wfmt == "f32":
        W = torch.from_numpy(synth.normal_f32((rows, cols), seed, 1, 0.0, std))
        return W, None, W.double()
    if wfmt == "bf16":
        W = torch.from_numpy(synth.normal_bf16((rows, cols), seed, 1, 0.0, std).view(np.int16)).view(torch.bfloat16)
        return W, None, W.double()
    if wfmt == "int8":
        q, s = synth.int8_rows(rows, cols, seed, 1, std)
        W, s = torch.from_numpy(q), torch.from_numpy(s)
        return W, s, W.double() * s.double()[:, None]
    block = 32 if wfmt == "int4" else 128
    q, s = synth.int4_blocks(rows, cols, seed, 1, std, block=block)
    W, s = torch.from_numpy(q), torch.from_numpy(s)
    code = torch.stack((W & 15, W >> 4), -1).flatten(-2).to(torch.int64)
    code = code - 16 * (code > 7)
    return W, s, code.double() * s.double().repeat_interleave(block, 1)


def rounded(a, dtype):
    return torch.as_tensor(a).to(dtype)


def sum_error(n, magnitude):
    return (n + STEPS) * U * magnitude


def widened_error(wfmt, x_is_bf16, magnitude, int4_parts):
    """int4 weights on the tensor cores are multiplied by their scale and rounded to bf16 where the
    batch is large (half a step of each weight), or to two bf16 parts (what the first leaves is
    half a step at most, and half a step of that is left out); 0 parts: every code is exact."""
    if wfmt in ("int4", "int4b128") and x_is_bf16 and int4_parts:
        return HALF[torch.bfloat16] ** int4_parts * magnitude
    return 0.0


def digit_error(x, Wd, wfmt):
    """bf16 tokens meet int8 and int4 weights as integers of 31 bits relative to the token's largest
    value m: each column is off by at most half a unit, 2^(e - 31) with 2^e <= 2 m."""
    if wfmt not in ("int8", "int4", "int4b128") or x.dtype != torch.bfloat16:
        return 0.0
    return 2.0 ** -30 * x.double().abs().amax(1, keepdim=True) * Wd.abs().sum(1)[None, :]


def linear(x, W, s_b, up=None, act_name="none", residual=None, y_dtype=torch.float32, wfmt="f32", int4_parts=0):
    """(reference, bound) of y = act(W x + b) [* (W_up x + b_up)] + residual; W, W_up float64
    [N, K]; s_b, and up's second entry: fp64 biases or None."""
    xd = x.double()
    bf = x.dtype == torch.bfloat16

    def product(Wd, b):
        v = xd @ Wd.T
        m = xd.abs() @ Wd.abs().T
        e = sum_error(Wd.shape[1], m) + widened_error(wfmt, bf, m, int4_parts) + digit_error(x, Wd, wfmt)
        if b is not None:
            v = v + b
            e = e + 2 * U * (v.abs() + b.abs())
        return v, e

    v, e = product(W, s_b)
    y = act(v, act_name)
    e = ACT_SLOPE * e + STEPS * U * y.abs()
    if up is not None:
        u, eu = product(*up)
        e = e * u.abs() + y.abs() * eu + e * eu
        y = y * u
    if residual is not None:
        y = y + residual.double()
        e = e + 2 * U * (y.abs() + residual.double().abs())
    return y, e + HALF[y_dtype] * (y.abs() + e) + TINY


def route(x, W_r, b, mask, k, router, scale):
    """Exact top k: (idx, w) with idx -1 / w 0 in slots that no selectable expert fills."""
    T, E = x.shape[0], W_r.shape[0]
    logits = x.double() @ W_r.double().T
    score = torch.sigmoid(logits) if router == "sigmoid" else logits
    key = score + (b.double() if b is not None and router == "sigmoid" else 0.0)
    idx = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros((T, k), dtype=torch.float64)
    for t in range(T):
        open_ = [e for e in range(E) if (mask is None or int(mask[e])) and math.isfinite(float(logits[t, e]))]
        best = sorted(open_, key=lambda e: (-float(key[t, e]), e))[:k]
        if not best:
            continue
        n = len(best)
        idx[t, :n] = torch.tensor(best, dtype=torch.int32)
        v = score[t, best] if router == "sigmoid" else torch.exp(score[t, best] - score[t, best].max())
        w[t, :n] = v / v.sum() * scale
    return idx, w


def ffn(x, gate, up, down, act_name):
    """(rows, bound) of one gated FFN over rows x (float64 weights)."""
    xd = x.double()
    H = gate.shape[1]
    g, u = xd @ gate.T, xd @ up.T
    eg = sum_error(H, xd.abs() @ gate.abs().T)
    eu = sum_error(H, xd.abs() @ up.abs().T)
    a = act(g, act_name)
    h = a * u
    ea = ACT_SLOPE * eg + STEPS * U * a.abs()
    eh = ea * u.abs() + a.abs() * eu + ea * eu
    eh = eh + 2.0 ** -16 * (h.abs() + eh) + TINY  # kept to 16 significant bits at least
    y = h @ down.T
    e = eh @ down.abs().T + sum_error(down.shape[1], (h.abs() + eh) @ down.abs().T)
    return y, e


def few(x, idx, w, experts, act_name, shared=None, residual=None):
    """(reference, bound) of the whole layer under the routing (idx, w)."""
    T, H = x.shape
    y = torch.zeros((T, H), dtype=torch.float64)
    e = torch.zeros((T, H), dtype=torch.float64)
    mag = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for j in range(idx.shape[1]):
            n = int(idx[t, j])
            if n < 0:
                continue
            r, er = ffn(x[t : t + 1], *(m[n] for m in experts), act_name)
            y[t] += float(w[t, j]) * r[0]
            e[t] += abs(float(w[t, j])) * er[0]
            mag[t] += abs(float(w[t, j])) * r[0].abs()
    terms = idx.shape[1]
    if shared is not None:
        r, er = ffn(x, *shared, act_name)
        y, e, mag, terms = y + r, e + er, mag + r.abs(), terms + 1
    if residual is not None:
        y, mag, terms = y + residual.double(), mag + residual.double().abs(), terms + 1
    e = e + sum_error(terms, mag + e)
    return y, e + HALF[x.dtype] * (y.abs() + e) + TINY


def check(got, ref, bound, what=""):
    got = got.detach().cpu().double()
    off = (got - ref).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), "%s: %d of %d values off; worst %.3g over its bound %.3g at %s" % (
        what, int(bad.sum()), bad.numel(), float((off - bound).nan_to_num(1e30).max()), float(bound.flatten()[
            int((off - bound).nan_to_num(1e30).argmax())]), np.unravel_index(int((off - bound).nan_to_num(1e30).argmax()), off.shape))
