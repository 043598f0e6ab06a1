"""ctypes declarations of libar_gb300.so (the C ABI in include/ar.h)."""

from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libar_gb300.so")

c_int, c_size_t, c_float, c_void_p = ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_void_p
VOIDPP = ctypes.POINTER(c_void_p)
SIZEP = ctypes.POINTER(c_size_t)
INTP = ctypes.POINTER(c_int)


class ArDesc(ctypes.Structure):
    _fields_ = [("n_ranks", c_int), ("count", c_size_t), ("dtype", c_int), ("algo", c_int),
                ("group_size", c_int), ("order", c_int), ("scale", c_float), ("collective", c_int),
                ("sm_budget", c_int), ("kernel", c_int), ("torus_dims", c_int * 3)]


class ArStats(ctypes.Structure):
    _fields_ = [("steps", c_int), ("launches", c_int), ("bytes_sent_per_rank", c_size_t),
                ("hbm_bytes", c_size_t), ("workspace_bytes", c_size_t)]


class ArFabric(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_double), ("bw_local", ctypes.c_double), ("bw_net", ctypes.c_double),
                ("ranks_per_server", c_int), ("in_network", c_int), ("shared_memory", c_int)]


class ArLogits(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("dtype", c_int), ("labels", c_void_p), ("temperature", c_float)]


class ArPolicyDesc(ctypes.Structure):
    _fields_ = [("clip_low", c_float), ("clip_high", c_float), ("kl_coef", c_float), ("mean", c_int),
                ("denominator", c_float), ("grad_scale", c_float)]


class ArPreferenceDesc(ctypes.Structure):
    _fields_ = [("beta", c_float), ("form", c_int), ("label_smoothing", c_float), ("target", c_float),
                ("length_normalized", c_int), ("denominator", c_float), ("grad_scale", c_float)]


class ArOrthoDesc(ctypes.Structure):
    _fields_ = [("n_matrices", c_int), ("rows", ctypes.POINTER(ctypes.c_int64)),
                ("cols", ctypes.POINTER(ctypes.c_int64)), ("in_dtype", c_int), ("out_dtype", c_int), ("steps", c_int),
                ("coefficients", ctypes.POINTER(c_float)), ("eps", c_float), ("precision", c_int)]


class ArMatrix(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("ld", ctypes.c_int64)]


class ArMuonDesc(ctypes.Structure):
    _fields_ = [("lr", c_float), ("momentum", c_float), ("weight_decay", c_float), ("nesterov", c_int),
                ("adjust", c_int), ("grad_scale", c_float)]


class ArTensor(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("count", ctypes.c_int64), ("dtype", c_int)]


class ArNormDesc(ctypes.Structure):
    _fields_ = [("kind", c_int), ("max_norm", ctypes.c_double), ("eps", ctypes.c_double), ("grad_scale", c_float)]


class ArAdamwDesc(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("grad_scale", c_float),
                ("step", ctypes.c_int64), ("device_step", c_void_p), ("device_lr", c_void_p)]


class ArScoreRows(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("rows", ctypes.c_int64), ("ld", ctypes.c_int64), ("dtype", c_int),
                ("temperature", c_float)]


class ArVerifyDesc(ctypes.Structure):
    _fields_ = [("target", ArScoreRows), ("draft", ArScoreRows), ("vocab", ctypes.c_int64), ("drafts", c_void_p),
                ("uniforms", c_void_p), ("draft_start", c_void_p), ("n_drafts", ctypes.c_int64),
                ("n_seq", ctypes.c_int64), ("mode", c_int)]


TENSORP = ctypes.POINTER(ArTensor)
MATRIXP = ctypes.POINTER(ArMatrix)

# name -> (restype, argtypes), in the order of include/ar.h
SIGNATURES = {
    "ar_plan": (c_int, [ctypes.POINTER(ArDesc), ctypes.POINTER(c_void_p)]),
    "ar_plan_stats": (c_int, [c_void_p, ctypes.POINTER(ArStats)]),
    "ar_plan_desc": (c_int, [c_void_p, ctypes.POINTER(ArDesc)]),
    "ar_execute": (c_int, [c_void_p, VOIDPP, VOIDPP, c_void_p, c_void_p]),
    "ar_execute_host": (c_int, [c_void_p, VOIDPP, VOIDPP, VOIDPP, c_void_p, c_void_p]),
    "ar_execute_noalloc": (c_int, [c_void_p, VOIDPP, VOIDPP, c_void_p]),
    "ar_bind": (c_int, [c_void_p, VOIDPP, VOIDPP, c_void_p, ctypes.POINTER(c_void_p)]),
    "ar_execute_bound": (c_int, [c_void_p, c_void_p]),
    "ar_bound_destroy": (None, [c_void_p]),
    "ar_plan_destroy": (None, [c_void_p]),
    "ar_plan_predict": (c_int, [c_void_p, ctypes.POINTER(ArFabric), ctypes.POINTER(ctypes.c_double)]),
    "ar_select": (c_int, [ctypes.POINTER(ArDesc), ctypes.POINTER(ArFabric), INTP, INTP,
                          ctypes.POINTER(ctypes.c_double)]),
    "ar_plan_transfers": (c_int, [c_void_p, c_int, INTP, INTP, ctypes.POINTER(ctypes.c_int64), c_int]),
    "ar_bucket_plan": (c_int, [SIZEP, c_int, c_size_t, c_size_t, INTP, INTP]),
    "ar_bucket_pack": (c_int, [c_int, VOIDPP, SIZEP, c_int, c_int, c_int, c_int, VOIDPP, c_void_p]),
    "ar_bucket_unpack": (c_int, [c_int, VOIDPP, c_float, c_int, VOIDPP, SIZEP, c_int, c_int, c_int,
                                 c_void_p]),
    "ar_bucket_allreduce": (c_int, [c_int, VOIDPP, SIZEP, c_int, c_int, c_int, c_int, c_float, c_int, c_int,
                                    c_void_p]),
    "ar_compress_sizes": (c_int, [c_size_t, c_int, SIZEP, SIZEP]),
    "ar_compress": (c_int, [c_int, c_size_t, c_int, c_int, VOIDPP, VOIDPP, VOIDPP, VOIDPP, c_void_p]),
    "ar_compressed_reduce": (c_int, [c_int, c_size_t, c_int, VOIDPP, VOIDPP, c_float, c_int, VOIDPP, c_void_p]),
    "ar_compressed_allreduce": (c_int, [c_int, c_size_t, c_int, c_int, VOIDPP, VOIDPP, c_float, VOIDPP,
                                        c_void_p]),
    "ar_token_logp": (c_int, [ctypes.POINTER(ArLogits), c_void_p, c_void_p]),
    "ar_loss_workspace": (c_int, [ctypes.c_int64, ctypes.c_int64, SIZEP]),
    "ar_policy_loss": (c_int, [ctypes.POINTER(ArLogits), c_void_p, c_void_p, c_void_p, c_void_p, ctypes.c_int64,
                               ctypes.POINTER(ArPolicyDesc), c_void_p, c_void_p, c_void_p, ctypes.c_int64, c_void_p,
                               c_void_p]),
    "ar_preference_loss": (c_int, [ctypes.POINTER(ArLogits), c_void_p, c_void_p, ctypes.c_int64,
                                   ctypes.POINTER(ArPreferenceDesc), c_void_p, c_void_p, c_void_p, c_void_p,
                                   ctypes.c_int64, c_void_p, c_void_p]),
    "ar_ortho_plan": (c_int, [ctypes.POINTER(ArOrthoDesc), ctypes.POINTER(c_void_p)]),
    "ar_ortho_plan_destroy": (None, [c_void_p]),
    "ar_ortho_workspace": (c_int, [c_void_p, SIZEP]),
    "ar_orthogonalize": (c_int, [c_void_p, MATRIXP, MATRIXP, c_void_p, c_void_p]),
    "ar_muon_step": (c_int, [c_void_p, ctypes.POINTER(ArMuonDesc), MATRIXP, MATRIXP, MATRIXP, MATRIXP, MATRIXP,
                             c_void_p, c_void_p]),
    "ar_muon_step_clipped": (c_int, [c_void_p, ctypes.POINTER(ArMuonDesc), MATRIXP, MATRIXP, MATRIXP, MATRIXP, MATRIXP,
                                     c_void_p, c_void_p, c_void_p]),
    "ar_grad_workspace": (c_int, [c_int, SIZEP]),
    "ar_grad_norm": (c_int, [TENSORP, c_int, ctypes.POINTER(ArNormDesc), c_void_p, c_void_p, c_void_p, c_void_p]),
    "ar_grad_clip": (c_int, [TENSORP, c_int, TENSORP, ctypes.POINTER(ArNormDesc), c_void_p, c_void_p, c_void_p,
                             c_void_p]),
    "ar_adamw_step": (c_int, [ctypes.POINTER(ArAdamwDesc), c_int, TENSORP, TENSORP, TENSORP, TENSORP, TENSORP,
                              TENSORP, TENSORP, TENSORP, TENSORP, c_void_p, c_void_p]),
    "ar_verify_workspace": (c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, SIZEP]),
    "ar_verify_drafts": (c_int, [ctypes.POINTER(ArVerifyDesc), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "ar_device_status": (c_int, [c_int]),
    "ar_plan_query": (c_int, [c_void_p]),
    "ar_selftest_wait_timeout": (c_int, [ctypes.c_uint, c_void_p]),
    "ar_selftest_scale_quotient": (c_int, [ctypes.POINTER(ctypes.c_ulonglong)]),
    "ar_status_string": (ctypes.c_char_p, [c_int]),
    "ar_version": (c_int, []),
}

_lib = None


def load() -> ctypes.CDLL:
    """Load the library; fail loudly if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python -m gradient_sync_gb300.build` "
                "(there is no fallback implementation)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def ptr_array(ptrs):
    arr = (c_void_p * max(1, len(ptrs)))()
    for i, p in enumerate(ptrs):
        arr[i] = p
    return arr
