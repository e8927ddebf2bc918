// append_axes.cu -- paged_kv_append_rope_axes: the instantiations of
// append_rope.cuh for positions of several axes.
//
// A lane's 4 cosines and sines come from up to 4 rows of the table, one 4-byte load
// each instead of two 16-byte ones; everything else is as there.  Bound by memory and
// by what waits for it (counts and axis positions, angles, with the rows beside
// them): 8 prompts of 900 to 2047 tokens, 64 + 8 heads of 128, bf16, three axes,
// norms 88 us, 82% of the copy rate (axis positions loaded when a token is known not
// to be padding: 92.5).
#include "append_rope.cuh"

namespace pa {

template <typename T, int D>
static cudaError_t launch_axes(const RopeAxesParams &p, cudaStream_t stream) {
    return p.pairs ? launch_mode<T, D, false, kNeighbours, true>(p, stream)
                   : launch_mode<T, D, false, kSplit, true>(p, stream);
}

template <typename T>
static cudaError_t launch_typed(int head_dim, const RopeAxesParams &p, cudaStream_t s) {
    switch (head_dim) {
        case 16:
            if constexpr (sizeof(T) == 4) return launch_axes<T, 16>(p, s);
            break;
        case 32: return launch_axes<T, 32>(p, s);
        case 64: return launch_axes<T, 64>(p, s);
        case 128: return launch_axes<T, 128>(p, s);
        case 256:
            if constexpr (sizeof(T) == 2) return launch_axes<T, 256>(p, s);
            break;
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_rope_append_axes(int dtype, int head_dim, const RopeAxesParams &p, cudaStream_t stream) {
    if (p.B == 0 || p.T == 0) return cudaSuccess;
    switch (dtype) {
        case PA_F32: return launch_typed<float>(head_dim, p, stream);
        case PA_F16: return launch_typed<__half>(head_dim, p, stream);
        case PA_BF16: return launch_typed<__nv_bfloat16>(head_dim, p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pa
