// answers.h -- answers of the CUDA runtime about a kernel, which stay the same while a
// process lives.  Host code only.
#pragma once

#include <mutex>

namespace edge {

// At most N answers, by kernel, size and device; more are asked for every time.
template <int N>
class Answers {
public:
    // The answer that is there, or ask()'s.  A negative one says that the question failed: it
    // is not kept, so the next call asks again.
    template <class Ask>
    int get(const void* fn, int size, int dev, Ask ask) {
        std::lock_guard<std::mutex> lock(mu_);
        for (int i = 0; i < used_; ++i) {
            if (table_[i].fn == fn && table_[i].size == size && table_[i].dev == dev) return table_[i].answer;
        }
        const int answer = ask();
        if (answer >= 0 && used_ < N) table_[used_++] = Entry{fn, size, dev, answer};
        return answer;
    }

private:
    struct Entry {
        const void* fn;
        int size, dev, answer;
    };
    std::mutex mu_;
    Entry table_[N];
    int used_ = 0;
};

}  // namespace edge
