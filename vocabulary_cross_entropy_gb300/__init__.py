"""GB300-native vocabulary cross entropy: a thin Python binding over libvce.so.

The functions here carry the names of the C ABI in ``include/vce.h`` and do
argument marshalling only: torch tensors supply device memory and the current
CUDA stream, every step of the computation runs in the library's sm_103a
kernels.  There is no CPU or PyTorch fallback: if libvce.so is missing or the
device is not a GB300 the calls raise.

Build the library with ``python -m vocabulary_cross_entropy_gb300.build``.
"""
from ._binding import (  # noqa: F401
    VceError,
    BF16,
    F32,
    DEVSTATUS_BAD_TARGET,
    DEVSTATUS_TIMEOUT,
    DEVSTATUS_BOUNDS,
    DEVSTATUS_BAD_ROW,
    DEFAULT_SLAB_BYTES,
    SLAB_UNCAPPED,
    REDUCE_NONE,
    REDUCE_MEAN,
    REDUCE_SUM,
    library,
    library_path,
    vce_status_string,
    vce_version,
    vce_kernel_launches,
    vce_bounds_check_build,
    ce_workspace_size,
    ce_forward,
    ce_forward_noalloc,
    ce_backward,
    ce_forward_backward,
    shift_targets,
    lce_workspace_size,
    lce_forward,
    lce_backward,
    selftest_lce_forward_timeout,
    selftest_ce_fused_timeout,
)
from ._head import (  # noqa: F401,E402
    MX_E4M3,
    MX_E2M1,
    SAMPLE_MAX_VOCAB,
    MXTensor,
    mx_codes_size,
    mx_scales_size,
    mx_quantize,
    mx_dequantize,
    mx_linear,
    rms_norm_forward,
    rms_norm_mx,
    rms_norm_workspace_size,
    rms_norm_backward,
    ce_sample,
    linear_sample,
)
from .autograd import parallel_cross_entropy, linear_cross_entropy, rms_norm  # noqa: F401,E402
