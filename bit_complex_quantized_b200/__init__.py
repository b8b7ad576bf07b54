"""B200-native PhaseQuant and multiplication-free complex GEMV/GEMM (libifq).

The compute path is the CUDA library libifq.so (include/ifq.h); this package
holds its ctypes binding (_lib), the in-tree build script (build) and the
seeded synthetic workload generator (workloads), and the host side of the
row split of a tensor across GPUs (shard).
"""
from ._lib import (  # noqa: F401
    EXPORTED,
    IFQ_DEV_NONFINITE,
    IFQ_DEV_RANGE,
    IFQ_DEV_TIMEOUT,
    IFQ_KV4_MAX_APPEND,
    IFQ_KV4_MAX_NEW,
    IFQ_MAX_GEMV_BATCH,
    IFQ_MAX_GROUP,
    IFQ_MAX_STAGES,
    IFQ_QUANT_STATIC_SCRATCH_BYTES,
    GemvPlan,
    IfqError,
    Kv4Cache,
    LayerSet,
    LIB_PATH,
    W4LayerSet,
    ifq_dequantize,
    ifq_gemm,
    ifq_gemm_wait_limit,
    ifq_gemv,
    ifq_gemv_workspace_bytes,
    ifq_kv4_append,
    ifq_kv4_attention,
    ifq_kv4_attention_workspace_bytes,
    ifq_kv4_read,
    ifq_quantize_pack,
    ifq_quantize_finish,
    ifq_quantize_pack_static,
    ifq_quantize_stage,
    ifq_quantize_workspace_bytes,
    ifq_status_string,
    ifq_w4_dequantize,
    ifq_w4_gemv,
    ifq_w4_quantize,
    ifq_widely_linear_from_real,
    ifq_widely_linear_quantize_pack,
    ifq_widely_linear_quantize_workspace_bytes,
    load,
    w4_shapes,
)
