// append_rope.cu -- paged_kv_append_rope and the 4-bit cache's appends: the
// instantiations of append_rope.cuh for positions of one axis.
#include "append_rope.cuh"

namespace pa {

template <typename T, int D, bool FP4>
static cudaError_t launch_one(const RopeAppendParams &p, cudaStream_t stream) {
    if (p.R == 0 || p.pairs) return launch_mode<T, D, FP4, kNeighbours>(p, stream);
    if constexpr (FP4) {
        if (p.R % 32 != 0) return launch_mode<T, D, FP4, kShuffle>(p, stream);
    }
    return launch_mode<T, D, FP4, kSplit>(p, stream);
}

bool rope_append_supported(int dtype, int head_dim) {
    if (dtype == PA_F32) return head_dim == 16 || head_dim == 32 || head_dim == 64 || head_dim == 128;
    return head_dim == 32 || head_dim == 64 || head_dim == 128 || head_dim == 256;
}

template <typename T>
static cudaError_t launch_typed(int head_dim, bool fp4, const RopeAppendParams &p, cudaStream_t s) {
    if (fp4) {
        switch (head_dim) {
            case 64: return launch_one<T, 64, true>(p, s);
            case 128: return launch_one<T, 128, true>(p, s);
            case 256: return launch_one<T, 256, true>(p, s);
        }
        return cudaErrorInvalidValue;
    }
    switch (head_dim) {
        case 16:
            if constexpr (sizeof(T) == 4) return launch_one<T, 16, false>(p, s);
            break;
        case 32: return launch_one<T, 32, false>(p, s);
        case 64: return launch_one<T, 64, false>(p, s);
        case 128: return launch_one<T, 128, false>(p, s);
        case 256:
            if constexpr (sizeof(T) == 2) return launch_one<T, 256, false>(p, s);
            break;
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_rope_append(int dtype, int head_dim, bool fp4, const RopeAppendParams &p, cudaStream_t stream) {
    if (p.B == 0 || p.T == 0) return cudaSuccess;
    switch (dtype) {
        case PA_F32: return launch_typed<float>(head_dim, fp4, p, stream);
        case PA_F16: return launch_typed<__half>(head_dim, fp4, p, stream);
        case PA_BF16: return launch_typed<__nv_bfloat16>(head_dim, fp4, p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pa
