"""fp32_gemm_amd -- single-precision GEMM for one AMD Instinct MI355X (gfx950).

C = alpha * A @ B + beta * C on row-major fp32 matrices, computed by the
hand-written HIP kernels of ``libfp32_gemm_amd.so`` behind a C ABI
(``include/fp32_gemm.h``).  The Python side only marshals arguments; PyTorch
supplies device memory and streams.

``include/grouped_gemm.h`` adds products grouped by expert with ragged sizes
(fp32, bf16, fp16), their weight gradient, and the product in 8-bit integers
with token and channel scales: ``gemm_grouped``, ``gemm_grouped_wgrad``,
``quantize_rows``, ``igemm``, and the product in microscaled 4-bit floats:
``quantize_mx4``, ``gemm_mx4``.

``include/layer_ops.h`` adds what stands around them in a layer: the
root-mean-square norm with a residual's addition and an 8-bit output, its
gradient, and a whole layer of experts for a few tokens: ``rms_norm``,
``rms_norm_grad``, ``expert_layer``.

The binding is loaded on first use of an API name, so ``fp32_gemm_amd.inputs``
can be imported on a machine where the library has not been built.
"""
_API = ("sgemm", "sgemm_ex", "sgemm_raw", "plan", "num_configs", "config_info", "configs",
        "status_string", "device_check", "SgemmError", "library_path", "check_tuple",
        "simulate_tuple", "exported_symbols", "tile_order", "ladder")
_GROUPED = ("gemm_grouped", "gemm_grouped_wgrad", "quantize_rows", "igemm", "quantize_mx4", "gemm_mx4",
            "GroupedGemmError")
_LAYERS = ("rms_norm", "rms_norm_grad", "expert_layer", "LayerError")


def __getattr__(name):
    if name == "binding" or name in _API:
        import importlib
        binding = importlib.import_module(__name__ + ".binding")
        return binding if name == "binding" else getattr(binding, name)
    if name == "grouped" or name in _GROUPED:
        import importlib
        grouped = importlib.import_module(__name__ + ".grouped")
        if name == "grouped":
            return grouped
        globals()[name] = getattr(grouped, name)  # found at once from the second use on
        return globals()[name]
    if name == "layers" or name in _LAYERS:
        import importlib
        layers = importlib.import_module(__name__ + ".layers")
        if name == "layers":
            return layers
        globals()[name] = getattr(layers, name)
        return globals()[name]
    raise AttributeError(name)


__all__ = list(_API + _GROUPED + _LAYERS)
