// kv_norm.hip -- fresh tokens into the paged cache with norms of their query
// and key heads ahead of the rotary positions (ptq1_kv_write_norm): the kernel
// of ptq1_kv_write (ptq1_kv_write.h), whose q and k rows lie in the registers
// of neighbouring lanes, so that a norm costs the exchanges of one sum and no
// more memory traffic than its gains.  HBM bounds it: 8191 tokens of 24 + 4 + 4
// heads of 256 (fp32 rows, bf16 queries and cache, 405 MB) take 96 us, 4.2 TB/s
// (the same rows without norms 87 to 91); one token 3.5 us on the GPU.
#include <hip/hip_runtime.h>

#include "ptq1_kv_write.h"

namespace ptq1 {

hipError_t launch_kv_write_norm(const void *q, int64_t qs, const void *k, int64_t ks, const void *v, int64_t vs, int src,
                                int64_t tokens, int32_t hq, const float *q_gain, const float *k_gain, float eps,
                                const int32_t *positions, const float *cos_sin, int64_t n_positions, int32_t rot,
                                const int64_t *slots, void *q_out, int q_type, const ptq1_kv_cache &c, hipStream_t s)
{
    KvWriteArgs a{q,     k,     v,         qs,          ks,        vs,        tokens, hq,
                  c.n_kv_heads, positions, cos_sin, n_positions, rot, slots, q_out, c.k_pages, c.v_pages,
                  c.k_steps, c.v_steps, c.n_pages * c.page_size, log2_of(c.page_size), 0, q_gain, k_gain, eps, 0, 0};
    return src == PTQ1_F32 ? write_q<true, float>(a, c.head_dim, c.dtype, q_type, s)
                           : src == PTQ1_F16 ? write_q<true, _Float16>(a, c.head_dim, c.dtype, q_type, s)
                                             : write_q<true, __bf16>(a, c.head_dim, c.dtype, q_type, s);
}

}  // namespace ptq1
