// tree_parts.h -- where the tree attention leaves the partial sums of a unit that
// lies in more than one run, and which of these entries the join may follow.  Plain
// C++, so that the rule can be checked on the host.
#pragma once

#ifdef __CUDACC__
#define STRATA_HD __host__ __device__ __forceinline__
#else
#define STRATA_HD inline
#endif

namespace strata {
namespace ta {

constexpr int MAX_CTAS = 148 * 2;           // CTAs (runs) the workspace has room for

// A run's first unit may have begun in an earlier run: slot 0; its last may go
// on in the next: slot 1.  Per unit: the run that begins it, and how many
// runs after that one go on with it.
struct Head {
  int run, follow;
};

// The slot of part i of a unit: slot 1 of the run that begins it, then slot 0 of the
// runs that go on with it.
STRATA_HD int part_slot(Head h, int i) { return 2 * (h.run + i) + (i == 0 ? 1 : 0); }

// Whether every part that the entry names is one of the workspace's 2 * MAX_CTAS
// slots.  A run that gave up a wait leaves the entries of its later units
// unwritten: they hold whatever the workspace held, and must not be followed.
// (No sum here can overflow, whatever the bytes are.)
STRATA_HD bool parts_within(Head h) {
  return h.run >= 0 && h.follow >= 0 && h.follow < MAX_CTAS && h.run < MAX_CTAS - h.follow;
}

}  // namespace ta
}  // namespace strata
