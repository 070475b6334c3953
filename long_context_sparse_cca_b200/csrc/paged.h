// Host-side launchers of the paged cache's kernels, called by the C ABI
// after it has checked every argument.
#pragma once

#include <cca.h>

#include "internal.h"

namespace cca {

// Workspace of a paged cache (byte offsets, 256-byte aligned).
struct PagedWorkspace {
    size_t tickets, part;                          // decode: arrivals, partial results
    size_t held;                                   // lengths at which rows were refused room
    size_t lens, old_held, flags, core_tmp, raw_tmp;  // fork: as they were, new tables
    size_t lists, counts;                          // fork, compact: page moves
    size_t total;
};
PagedWorkspace paged_workspace(const cca_paged_cache &c);

size_t paged_decode_part_bytes(const cca_paged_cache &c);
cudaError_t launch_paged_decode(const cca_paged_cache &c, int layer, const void *q_t,
                                const void *k_t, const void *v_t, void *o_t, bool o_f32,
                                void *workspace, cudaStream_t s);
cudaError_t launch_paged_fill(const cca_paged_cache &c, int layer, const PackedRows &K,
                              const PackedRows &V, const void *Kc, const void *Vc, const int *cu,
                              const int *rows, int S, int64_t total, cudaStream_t s);
cudaError_t launch_paged_reserve(const cca_paged_cache &c, const long long *n_new, long long n,
                                 void *workspace, cudaStream_t s);  // workspace: NULL: no marks
cudaError_t launch_paged_fork(const cca_paged_cache &c, const int *parent, void *workspace,
                              cudaStream_t s);
cudaError_t launch_paged_compact(const cca_paged_cache &c, long long *live, void *workspace,
                                 cudaStream_t s);
cudaError_t paged_decode_status_read_clear(unsigned int *v);
cudaError_t paged_tables_status_read_clear(unsigned int *v);

}  // namespace cca
