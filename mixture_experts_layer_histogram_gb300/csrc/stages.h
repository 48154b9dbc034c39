// The way of a reader warp through the stages of its block's ring, on the GPU and (in a test) on the host.
//
// The block's reader warps take `total` stages each and meet after every `per_group` of them (a multiple of which `total` is), at
// barriers that count all of them. A warp whose wait gives up therefore goes on to every meeting, without waiting for or using
// another stage: one that left would keep those that saw the same stage land just in time at the barrier for good.
#pragma once

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

// wait(i): whether stage i has come (false: given up), the same for all lanes of a warp; use(i) takes it; meet(ok): the barriers,
// ok: this warp has taken every stage. Returns ok at the end.
template <typename Wait, typename Use, typename Meet>
MOE_HOST_DEVICE bool through_stages(int total, int per_group, const Wait &wait, const Use &use, const Meet &meet) {
  bool ok = true;
  for (int i = 0, k = 0; i < total; ++i) {
    if (ok) ok = wait(i);
    if (ok) use(i);
    if (++k < per_group) continue;
    k = 0;
    meet(ok);
  }
  return ok;
}

}  // namespace moe
