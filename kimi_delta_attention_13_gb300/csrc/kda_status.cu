// kda_status.cu -- the translation units' sticky error words, read and cleared in one pass: a thread exchanges each
// with 0, so that no error that another stream's kernel raises meanwhile is lost, and one copy and one wait bring
// the first to the host.  (A copy, a clearing and a wait a word took 192 us for nine words, this 36.)
#include <mutex>

#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kWords = 9;
struct Words {
    int *at[kWords];   // in the order of which one is told first
};

__device__ int g_first_error;   // what the host copies

__global__ void status_kernel(const Words w)
{
    const int lane = threadIdx.x;
    const int e = lane < kWords ? atomicExch(w.at[lane], 0) : 0;
    const unsigned set = __ballot_sync(0xffffffffu, e != 0);
    const int first = __shfl_sync(0xffffffffu, e, set ? __ffs(set) - 1 : 0);
    if (lane == 0) g_first_error = first;
}

}  // namespace

int read_and_clear_status(cudaStream_t s, int32_t *status)
{
    static std::mutex one;   // a device has one g_first_error
    const std::lock_guard<std::mutex> lock(one);
    const Words w = {{status_word_prefill_tc(), status_word_prefill_tc_precise(), status_word_decode(), status_word_cp(),
                      status_word_linear(), status_word_delta(), status_word_delta_decode(), status_word_state_copy(),
                      status_word_state_pack()}};
    for (int *p : w.at)
        if (!p) return KDA_ERR_CUDA;
    status_kernel<<<1, 32, 0, s>>>(w);
    int host = 0;
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyFromSymbolAsync(&host, g_first_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return KDA_ERR_CUDA;
    *status = host;
    return KDA_OK;
}

}  // namespace kda
