// The paged attention kernel for MXFP4 caches (one E8M0 scale per 32 channels).
#include "paged_attn.cuh"

namespace csa2 {

int paged_attn_mx_wait_flag(bool clear) { return read_device_flag(pa::g_paged_attn_error, clear); }

int pa::launch_paged_attn_mxfp4(const Args &a, int nh, int G, cudaStream_t s) { return launch_attn<true>(a, nh, G, s); }

}  // namespace csa2
