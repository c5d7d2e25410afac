"""GB300-native (sm_103a) TMA-pipelined fp16 GEMM  C = A . B^T.

The GEMM is the C-ABI library ``libtmagemm.so`` (declared in
``include/tmagemm.h``, built by ``build.py`` from ``csrc/``); ``binding``
exposes its entry points under the same names.  ``inputs`` generates the
seeded synthetic operands used by the tests and the benchmark.

``experts`` adds the operators of an expert layer around the GEMM (declared in
``include/tmaexperts.h``): ``ExpertRoute`` (tokens sorted by expert and back),
``GroupedPlan`` (the experts' products) and ``W4Plan`` (products with 4-bit
weights).

``microscale`` adds block-scaled 8- and 4-bit floating point (declared in
``include/tmamicro.h``): ``mx_quantize``, ``MXTensor`` and ``MXPlan`` (their products).
``layer`` adds what surrounds the products (declared in ``include/tmalayer.h``):
``rms_norm``, ``rms_norm_grad``, ``GradClip`` and ``clip_grad_norm``.
"""
from .binding import (  # noqa: F401
    GEMM_OUT_F16, GEMM_OUT_F32, GemmError, Plan, VARIANTS, gemm_create_plan,
    gemm_create_plan_ex, gemm_destroy, gemm_get_device_status, gemm_last_error,
    gemm_last_status, gemm_plan_config, gemm_plan_describe, gemm_run, gemm_run_host,
    gemm_schedule_tile, gemm_select_config, gemm_sw128_offset, make_options)
from .experts import ExpertRoute, GroupedPlan, W4Plan, w4_pack  # noqa: F401
from .layer import GradClip, clip_grad_norm, rms_norm, rms_norm_grad  # noqa: F401
from .microscale import MXPlan, MXTensor, mx_quantize  # noqa: F401
