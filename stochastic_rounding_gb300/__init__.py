"""GB300-native fused AdamW step with Philox-keyed stochastic rounding to bf16.

The computation lives in ``libasr.so`` (CUDA kernels for sm_103a behind a C
ABI, declared in ``include/asr.h``); this package is its ctypes binding plus
the synthetic workload definitions used to exercise it.
"""
from ._lib import (  # noqa: F401
    ASR_BF16, ASR_F32, ASR_ROUND_RNE, ASR_ROUND_SR, AsrError, asr_adamw_prepare,
    asr_adamw_sr_multi_tensor, asr_adamw_sr_multi_tensor_static, asr_adamw_sr_step,
    asr_gemm_bf16_sr, asr_last_cuda_error, asr_philox4x32, asr_status_string,
    asr_stochastic_round_bf16, asr_take_device_error, asr_take_device_error_async, asr_selftest_wait_timeout,
    asr_kernel_launches, asr_adamw_sr_multi_tensor_host, lib, make_host_table, make_table,
    asr_gemm_int8_sr, asr_gemm_int8_workspace, asr_muon_sr_multi_tensor, asr_muon_workspace, asr_newton_schulz,
    asr_newton_schulz_workspace, asr_quantize_int8, int8_empty, asr_linear_int8, asr_linear_int8_workspace,
    asr_linear_int8_grads, asr_linear_int8_grads_workspace, asr_checkpoint_int8, asr_restore_int8, asr_activation,
    asr_activation_grads, asr_layer_norm, asr_layer_norm_grads, asr_layer_norm_grads_workspace, asr_embedding,
    asr_embedding_grads, asr_embedding_grads_workspace,
)
from .int8 import (Int8Checkpoint, Int8Linear, checkpoint_int8, int8_linear, int8_linear_grads,  # noqa: F401,E402
                   restore_int8)
from .layers import (Activation, Embedding, LayerNorm, NormSaved, activation, activation_grads,  # noqa: F401,E402
                     embedding, embedding_grads, layer_norm, layer_norm_grads)
from .optim import AdamWSR, DeviceError  # noqa: F401,E402
from .muon import MuonSR  # noqa: F401,E402
