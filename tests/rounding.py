"""Comparison of rounded outputs: a kernel that computes v with |v - ref| <= tol and rounds it once, to
nearest, returns a value between the roundings of ref - tol and ref + tol (rounding is monotone). For
fp32 outputs the tolerance itself holds their rounding."""
import numpy as np
import torch


def round_to(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, np.float64)).to(torch.float32).to(dtype).double().numpy()


def within_one_rounding(got, ref, tol, dtype):
    """`got` (float64, of outputs of `dtype`) is one rounding of values within `tol` of `ref`."""
    if dtype == torch.float32:
        return bool((np.abs(got - ref) <= tol).all())
    return bool(((got >= round_to(ref - tol, dtype)) & (got <= round_to(ref + tol, dtype))).all())
