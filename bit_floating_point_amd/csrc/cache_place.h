// Where a position of a sequence lies in a cache, from what the host cannot check: page tables,
// positions and sequence numbers of any content.  Plain integers, no GPU.
#pragma once
#include <stdint.h>

#if defined(__HIPCC__)
#define FP4_HD __host__ __device__
#else
#define FP4_HD
#endif

namespace fp4 {

// the page that an entry of the table names, -1 if the cache has no such page
FP4_HD inline int32_t page_at(const int32_t* entry, int32_t pages) {
    const int32_t page = *entry;
    return (uint32_t)page < (uint32_t)pages ? page : -1;
}

struct RowPlace {
    int32_t page, slot;  // page -1: no row
};
// the row of `position` of `sequence`; `capacity`: positions that a row of the table has pages for
FP4_HD inline RowPlace find_row(const int32_t* table, int64_t sequences, int64_t ld, int32_t capacity, int32_t page_log, int32_t pages,
                                int64_t sequence, int32_t position) {
    if ((uint64_t)sequence >= (uint64_t)sequences || (uint32_t)position >= (uint32_t)capacity) return RowPlace{-1, 0};
    return RowPlace{page_at(table + sequence * ld + (position >> page_log), pages), position & ((1 << page_log) - 1)};
}

}  // namespace fp4
