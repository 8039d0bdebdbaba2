"""libflce: chunked fused LM-head cross-entropy on GB300 (sm_103a).

The compute lives in the C-ABI CUDA library (include/flce.h, csrc/); this
package holds its ctypes binding, a thin torch-facing API and the seeded
synthetic workloads.
"""
from .api import (IGNORE_INDEX, DistillLoss, GRPOLoss, LinearCrossEntropy,  # noqa: F401
                  LinearCrossEntropyLoss, SelectiveLogSoftmax,
                  backward, distill_loss, forward, forward_backward, grpo_loss, grpo_token_loss,
                  jsd_backward, jsd_forward, kd_backward, kd_forward, linear_cross_entropy,
                  scale_grads, selective_log_softmax, workspace_bytes)
from .layer_norm import LayerNorm, layer_norm, layer_norm_backward, layer_norm_forward  # noqa: F401
from .norm import (RMSNorm, RMSNormFunction, rms_norm, rms_norm_backward, rms_norm_e4m3,  # noqa: F401
                   rms_norm_forward)
from .score import (score_backward, score_forward, selective_log_softmax_entropy,  # noqa: F401
                    top_logprobs)
from .topk import (TopkDistill, TopkDistillOneCall, topk_distill_loss, topk_kd_backward,  # noqa: F401
                   topk_kd_forward, topk_kd_forward_backward)
