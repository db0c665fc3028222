// ddp_spans.h -- spans of memory and pointers, as the entry points check them.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <iterator>
#include <utility>
#include <vector>

#include "ddp.h"

namespace ddpk {

using Span = std::pair<uintptr_t, uintptr_t>;      // [first, second) in bytes

inline Span span_of(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + (uintptr_t)bytes};
}

// Sorts the spans; true if two of them share a byte.
inline bool any_overlap(std::vector<Span>* v) {
    std::sort(v->begin(), v->end());
    for (size_t i = 1; i < v->size(); ++i)
        if ((*v)[i].first < (*v)[i - 1].second) return true;
    return false;
}

// Sorts the spans and joins those that share a byte or touch.
inline void unite(std::vector<Span>* v) {
    std::sort(v->begin(), v->end());
    size_t n = 0;
    for (const Span& s : *v) {
        if (n > 0 && s.first <= (*v)[n - 1].second) (*v)[n - 1].second = std::max((*v)[n - 1].second, s.second);
        else (*v)[n++] = s;
    }
    v->resize(n);
}

// True if s shares a byte with one of the sorted, disjoint spans.
inline bool hits_any(const std::vector<Span>& sorted, Span s) {
    auto it = std::lower_bound(sorted.begin(), sorted.end(), Span{s.second, 0});
    return it != sorted.begin() && std::prev(it)->second > s.first;
}

inline int32_t check_ptr(const void* p, int64_t align) {
    if (!p) return DDP_ERR_INVALID;
    return reinterpret_cast<uintptr_t>(p) % (uintptr_t)align ? DDP_ERR_ALIGN : DDP_OK;
}

}  // namespace ddpk
