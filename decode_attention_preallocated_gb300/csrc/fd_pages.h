// fd_pages.h -- launchers of the page bookkeeping of a paged cache
// (fd_pages.cu): reference-counted pages, a block table and lengths, all on
// the device.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fd {

struct Books {
    int32_t *table;        // [B, max_pages]
    int32_t *lengths;      // [B]
    int32_t *refs;         // [num_pages]: table entries that name the page
    int32_t B, max_pages, page_size, num_pages;
    int32_t *status;
};

constexpr int kMaxPools = 256;

// Pools whose pages are copied together: page i of pool q is the bytes[q]
// bytes at base[q] + i * step[q].  units[q] is the first of pool q's copy
// units within a page, units[n] their number.
struct Pools {
    uint8_t *base[kMaxPools];
    int64_t step[kMaxPools];
    int64_t bytes[kMaxPools];
    int32_t units[kMaxPools + 1];
    int32_t n;
};
int pages_unit_bytes();

// Scratch that reserve and compact want, in int32 words.
int64_t pages_scratch_words(int64_t num_pages);

int launch_pages_free(const Books &k, const int32_t *seqs, const int32_t *lengths, int n,
                      cudaStream_t st);
int launch_pages_fork(const Books &k, const int32_t *src, const int32_t *dst,
                      const int32_t *lengths, int n, cudaStream_t st);
// Rows that one block of the reordering holds a column of.
constexpr int kReorderRows = 49152;
int launch_pages_reorder(const Books &k, const int32_t *src, int32_t *ticket, cudaStream_t st);
int launch_pages_reserve(const Books &k, const int32_t *n_new, int n_each, int32_t *pairs,
                         int32_t *count, int32_t *scratch, cudaStream_t st);
int launch_pages_compact(const Books &k, int32_t *pairs, int32_t *count, int32_t *scratch,
                         cudaStream_t st);
int launch_pages_copy(const Pools &q, const int32_t *pairs, const int32_t *count, int max_pairs,
                      int num_pages, int32_t *status, int sms, cudaStream_t st);

}  // namespace fd
