"""Which kernel a block-scaled product goes to (not a test module)."""
import ctypes

ACTS = {None: 3, "tanh": 0, "erf": 1, "relu": 2}
OUTS = {"f32": 0, "bf16": 1, "e4m3": 2}
B200_SMS = 148


def few_rows(rm, G, M, N, K, out, act=None, sms=B200_SMS):
    """True: the few-row kernel, False: the CTA pairs."""
    a = rm.rm_matmul_fp8_args(G=G, M=M, N=N, K=K, w_block_rows=128, act=ACTS[act], out_dtype=OUTS[out])
    return bool(rm._lib.rm_internal_matmul_fp8_few_rows(ctypes.byref(a), sms))
