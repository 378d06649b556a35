"""How near an attention of fp32 operands in two f16 parts comes, and what a lost part costs."""
import numpy as np

# Of the output's root mean square: four times the 2^-20 to which a plain fp32 form's sums come
# (0.4 to 1.0e-6 over 100 to 8000 keys), for two parts hold a number to 2^-22 and the tensor cores
# cut their fp32 sums.  A number in one part of 11 bits is off by up to 2^-12 of its binade, 2^-12.8
# in the mean square.
LIMIT = 2.0 ** -18


def rms(got, want):
    """The error's root mean square in units of the output's."""
    return float(np.sqrt(np.mean((got - want) ** 2) / np.mean(want ** 2)))


def parts(x, low=True):
    """x in f16 parts of a scale that takes each row's largest value into [2^14, 2^15)."""
    top = np.abs(x).max(-1, keepdims=True)
    scale = 2.0 ** (14 - np.floor(np.log2(np.where(top == 0, 1, top))))
    high = (x * scale).astype(np.float16).astype(np.float64)
    rest = (x * scale - high).astype(np.float16).astype(np.float64) if low else 0 * high
    return high / scale, rest / scale


def product(a, b, low_a=True, low_b=True):
    """a b^T of rows in two parts each, low x low left out."""
    ah, al = parts(a, low_a)
    bh, bl = parts(b, low_b)
    return ah @ bh.T + ah @ bl.T + al @ bh.T


def attend(q, k, v, scale, lost=""):
    """softmax(scale q k^T) v, the low parts of the operands in `lost` dropped."""
    x = product(q, k, "q" not in lost, "k" not in lost) * scale
    p = np.exp(x - x.max(-1, keepdims=True))
    vh, vl = parts(v, "v" not in lost)
    ph, pl = parts(p, "p" not in lost)
    return (ph @ vh + ph @ vl + pl @ vh) / p.sum(-1, keepdims=True)
