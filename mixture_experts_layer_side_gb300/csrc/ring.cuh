// Fills of a ring of stages, counted from 0: fill f goes to stage f % stages,
// whose mbarrier then completes its phase number f / stages.
#pragma once

#ifndef __CUDACC__
#define __host__
#define __device__
#endif

namespace mok {

// The parity to wait for, for fill f to have landed.
__host__ __device__ constexpr unsigned fill_parity(int f, int stages) { return (unsigned)(f / stages) & 1u; }

// Of `issued` fills, the first that no later one of its stage followed: the fills from it on are each their stage's last.
// Those before landed before their stage was filled again.
__host__ __device__ constexpr int last_fills_from(int issued, int stages) { return issued > stages ? issued - stages : 0; }

}  // namespace mok
