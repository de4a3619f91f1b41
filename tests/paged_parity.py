"""Comparison of the paged attention kernels with the oracle, per element and in the norm.

A row's result may be off from its 64-bit value by
  2^-8 |ref| + (2^-8 + 2^-18) spread + 2^-25 share + (e^(2 delta) - 1) apart                        (per element)
with spread = sum_j p_j |v_j|, share = max_j p_j sum_j |v_j| and apart = sum_j p_j |v_j - ref|, all over the keys that
this row sees and no others:
  * 2^-8 |ref|: out is rounded to bf16 (half a step);
  * 2^-8 spread: a probability enters its product with 8 significant bits or more (half a step);
  * 2^-25 share: or with an error of at most 2^-25 of the row's largest one, if that is more;
  * 2^-18 spread: the exponential and the row sum, 2^-19 each;
  * delta = (d + 16) 2^-24 mass: a score is a sum of d fp32 products, whose magnitudes add up to mass. Scores that are
    off by up to delta change p_j by factors of e^(+-2 delta) after the division, and only differences between the
    values matter then.
The roundings of different p_j are independent and centred, so the squares of the first two terms add up: over all
elements of a call the 2-norm of the error is at most that of
  2 sqrt((2^-8 ref)^2 + 2^-16 sum_j p_j^2 v_j^2) + the last three terms,
where the factor 2 is for a sum of few terms, and half steps are twice the root mean square of a rounding already.
lse may be off by delta + 2^-19 + 2^-22 |ref|.
"""
import numpy as np

from oracle import paged as op


def expected(q, cache, table, q_start, kv_len, causal, max_kv=None):
    """Everything that `check` compares with, from numpy arrays."""
    out, lse, spread, mass = op.attention(q, cache, table, q_start, kv_len, causal, max_kv)
    square, share, apart, others = op.attention_weights(q, cache, table, q_start, kv_len, causal, max_kv)
    delta = (q.shape[-1] + 16) * 2.0 ** -24 * mass
    rest = 2.0 ** -18 * spread + 2.0 ** -25 * share + np.expm1(2 * delta)[..., None] * apart
    return {"out": out, "lse": lse, "most": 2.0 ** -8 * (np.abs(out) + spread) + rest,
            "norm": 2 * np.sqrt((2.0 ** -8 * out) ** 2 + 2.0 ** -16 * square) + rest,
            "others": others, "lse_most": delta + 2.0 ** -19 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))}


def roundings(want):
    """The 2-norm that the error of a call's result has if nothing is rounded but out, and each probability but its row's
    largest to 8 bits: steps of s leave s^2 / 12 each, relative roundings within +-2^-9 leave p^2 2^-18 / 3. Over many
    rows an error's norm stays within a few hundredths of it."""
    ref = want["out"][~np.isnan(want["out"][:, 0, 0])]
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(ref), 1e-30))) - 7)
    return np.sqrt(np.sum(step ** 2) / 12 + np.sum(want["others"]) * 2.0 ** -18 / 3)


def problems(out, lse, want):
    """What is wrong with out [T, Hq, d] and lse [T, Hq] (fp64 numpy, lse may be None), as a list of texts."""
    rows = ~np.isnan(want["out"][:, 0, 0])
    ref, got = want["out"][rows], out[rows]
    found = []
    with np.errstate(invalid="ignore", over="ignore"):
        err = np.abs(got - ref)
        over = ~(err <= want["most"][rows])                       # NaN counts as wrong
        if over.any():
            at = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err / np.maximum(want["most"][rows], 1e-300))), err.shape)
            found.append(f"{over.sum()} of {over.size} elements off, worst at {at}: {got[at]} for {ref[at]} +- {want['most'][rows][at]}")
        norm, lim = np.sqrt(np.sum(err ** 2)), np.sqrt(np.sum(want["norm"][rows] ** 2))
        if not norm <= lim:
            found.append(f"norm of the error {norm}, at most {lim}")
        if lse is not None:
            ref, got = want["lse"][rows], lse[rows]
            same = (ref == got) | (np.abs(got - ref) <= want["lse_most"][rows])
            if not same.all():
                found.append(f"{(~same).sum()} of {same.size} lse off")
    return found


def check(out, lse, want):
    f64 = lambda t: None if t is None else t.detach().cpu().double().numpy()  # noqa: E731
    found = problems(f64(out), f64(lse), want)
    assert not found, "; ".join(found)
