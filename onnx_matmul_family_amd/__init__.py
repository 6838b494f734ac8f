"""ONNX MatMul-family operators for AMD Instinct MI355X (gfx950).

MatMul, Gemm, QLinearMatMul and GroupedMatMul, and around them the operators
of a language model's decode step (a projection with per-row low-rank
adapters, the expert router, the expert layer of a few tokens, token log
probabilities and their gradient), as hand-written HIP kernels
behind the C ABI in include/omm.h (libomm.so); this package is the thin
Python binding (`_omm`), the build step (`build`) and the seeded input
generators (`synth`).  The binding is imported lazily so that the generators
and the build step work on machines without a GPU.
"""

_BINDING = ("matmul", "gemm", "gemm_noalloc", "qlinear_matmul", "grouped_matmul", "grouped_matmul_dequant",
            "grouped_matmul_check", "grouped_matmul_workspace_size", "describe", "lib", "status_string", "OmmError",
            "OmmTensor", "lora_matmul", "lora_matmul_workspace_size", "moe_route", "moe_layer",
            "moe_layer_workspace_size", "token_logprobs", "token_logprobs_workspace_size", "token_logprobs_grad")


def __getattr__(name):
    if name in _BINDING:
        from . import _omm
        value = globals()[name] = getattr(_omm, name)  # (found without this function from now on)
        return value
    raise AttributeError(name)
