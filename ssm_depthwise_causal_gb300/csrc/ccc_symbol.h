// ccc_symbol.h -- the address of a device variable in the current context,
// looked up once a context.
#pragma once

#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

namespace ccc {

// Unique ID of the context current on this thread, which the driver never
// reuses within a process; 0 when there is none yet (or it cannot be read).
unsigned long long current_context_id();

class SymbolAddress {
  public:
    // symbol: the variable's address as host code takes it.  Null where the lookup fails.  Without a context it makes the current
    // device's primary context current, as any runtime call would.
    void *find(const void *symbol) {
        const auto look = [&] {
            void *p = nullptr;
            if (cudaGetSymbolAddress(&p, symbol) == cudaSuccess) return p;
            cudaGetLastError();  // (told by the null)
            return static_cast<void *>(nullptr);
        };
        unsigned long long id = current_context_id();
        if (id == 0) {
            void *p = look();
            id = p ? current_context_id() : 0;
            if (id == 0) return p;  // cannot key it: the fresh lookup, uncached
        }
        std::lock_guard<std::mutex> lock(mu_);
        for (const Entry &e : cache_)
            if (e.ctx_id == id) return e.addr;
        void *p = look();
        if (p) {
            cache_[next_] = Entry{id, p};
            next_ = (next_ + 1) % kEntries;
        }
        return p;
    }

  private:
    struct Entry {
        unsigned long long ctx_id;
        void *addr;
    };
    static constexpr int kEntries = 64;
    std::mutex mu_;
    Entry cache_[kEntries] = {};
    int next_ = 0;
};

}  // namespace ccc
