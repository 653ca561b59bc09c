"""64-bit forms of the rotations of a qkv_rope, written pair by pair, and the bound of their error.

Error of a turned value (u = 2^-24): the angle, in half turns of size at most 1, is off by half a step of f32, 2^-25,
and by 2^-32 from the cut to 32 bits: 1.6 u of an angle.  sincospi is off by at most one unit in the last place, u for a
value below 1, and the magnitude rounds once more: 3.6 u of the magnitude.  Two products and a sum round once each:
|r - exact| <= 6 u magnitude (|x0| + |x1|), taken as 7 u.  Then one rounding to the output's type.
"""
import math

import numpy as np

U = 2.0 ** -24
HALF_STEP = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def freqs(rot, theta, scaling="none", factor=1.0, orig_ctx=0.0, low=0.0, high=0.0, divisors=None, **_):
    out = []
    for d in range(rot // 2):
        base = theta * factor ** (rot / (rot - 2)) if scaling == "base" else theta
        f = base ** (-2 * d / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "table":
            f /= divisors[d]
        if scaling == "ramp":
            first = max(0, math.floor(rot / 2 * math.log(orig_ctx / (high * 2 * math.pi), theta)))
            last = min(rot - 1, math.ceil(rot / 2 * math.log(orig_ctx / (low * 2 * math.pi), theta)))
            g = 0.0 if d <= first else 1.0 if d >= last else (d - first) / (last - first)
            f = g * f / factor + (1 - g) * f
        if scaling == "bands":
            turns = orig_ctx * f / (2 * math.pi)
            if turns <= low:
                f /= factor
            elif turns < high:
                g = (turns - low) / (high - low)
                f = (1 - g) * f / factor + g * f
        out.append(f)
    return np.array(out)


def pairs(rot, neighbours):
    d = np.arange(rot // 2)
    return (2 * d, 2 * d + 1) if neighbours else (d, d + rot // 2)


def turn(x, pos, f, rot, neighbours, magnitude=1.0, inverse=False):
    """x [nt, heads, hd] in 64 bits; the turned values and the bound of their f32 errors."""
    a, b = pairs(rot, neighbours)
    angle = (np.asarray(pos, np.float64)[:, None] * f)[:, None]
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle) * (-1 if inverse else 1)
    r, bound = x.astype(np.float64).copy(), np.zeros(x.shape)
    r[..., a] = x[..., a] * c - x[..., b] * s
    r[..., b] = x[..., a] * s + x[..., b] * c
    size = 7 * U * magnitude * (np.abs(x[..., a]) + np.abs(x[..., b])) + 1e-37
    bound[..., a], bound[..., b] = size, size
    return r, bound


def rounded(bound, value, dtype):
    """The bound with the rounding to dtype added (f16 has subnormals of 2^-24)."""
    step = HALF_STEP[dtype] * (np.abs(value) + bound)
    if dtype == "f16":
        step = np.maximum(step, 2.0 ** -25)
    return bound + (step if dtype != "f32" else 0.0)


FORMS = [dict(scaling="none"), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
         dict(scaling="ramp", factor=4.0, orig_ctx=32768.0, low=1.0, high=32.0, magnitude=1.1386),
         dict(scaling="bands", factor=8.0, orig_ctx=8192.0, low=1.0, high=4.0), dict(scaling="table")]


def create(Q, hd, rot, neighbours, theta, form):
    """The framework's rope of a form, and its reference frequencies."""
    form = dict(form)
    if form["scaling"] == "table":
        form["divisors"] = [1.0 + 0.25 * d for d in range(rot // 2)]
    kind = ["none", "linear", "base", "ramp", "bands", "table"].index(form["scaling"])
    rope = Q.qkv_rope_create(hd, theta, rot_dim=rot, layout=Q.QKV_ROPE_INTERLEAVED if neighbours else Q.QKV_ROPE_NEOX,
                             **{**form, "scaling": kind})
    return rope, freqs(rot, theta, **form)
